// kv_append.cu -- new keys and values into a paged cache, the keys rotated on
// the way and, where given, the queries of the same tokens with them.
//
// Token i of sequence b goes to position p = past_lens[b] + i: row
// p % page_size of page block_table[b][p / page_size].  Keys (and queries) are
// turned by the angles of p, then rounded once to the cache's type; an 8-bit
// cache holds x / scale[head], rounded to the nearest e4m3 and saturated.
//
// Memory bound, and at one token a sequence bound by latency: the heads of a
// token (queries, keys, values, in this order) are one list, a thread owns a
// column unit of one token for a run of that list, so one launch does all
// three tensors, and position, page and angles are found once per thread.  The
// first heads are loaded before position and page are known, and queries, keys
// and values are walked by loops of their own (one loop that chose the tensor
// head by head took 138 us below).
//
// Measured on a GB300: a 32K prompt of 32 query and 8 + 8 key and value heads
// of 128, straight from a fused projection: 122 us, 98 % of the measured copy
// bandwidth; one token of 32 sequences: 3.0 us; 6 x 1000 padded tokens of 24
// heads of 64 into an 8-bit cache: 8.2 us, bound by the latency of short
// threads (3 us of bytes).
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "quantize4.cuh"
#include "rotate.cuh"

namespace mercury {

// Error word of this file's kernel: kPagedErrBounds = a token's position or
// page lies outside the table or the cache and was not written; the first
// site (0x801 new_lens, 0x802 position, 0x803 page).
__device__ unsigned int g_append_err_word = 0;
__device__ unsigned int g_append_err_site = 0;

namespace {

__device__ __noinline__ void record_bounds(unsigned int site)
{
    atomicOr(&g_append_err_word, kPagedErrBounds);
    atomicCAS(&g_append_err_site, 0u, site);
}

struct AppendArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out;
    Strides qs, ks, vs, os;
    const int *past, *new_lens;
    PagedView cache;
    int Hq, S, d, head_groups, heads_per_thread, units, tokens_per_block;
    long long tokens;
    int copy_rest;  // q_out is not q itself
    mercury_rope_plan plan;
};

template <bool T>
struct Turn {
    static constexpr bool value = T;
};

// One head's unit (two chunks of 8 of 16-byte accesses, as loaded) into a row of
// a 4-bit cache.  The chunks of a unit of the rotated part (turned or, of values,
// not) are halves of two blocks, whose other halves the neighbouring lane has;
// any other unit's make one block.
template <bool TURN>
__device__ __forceinline__ void keep4(const RotUnit<8> &unit, const mercury_rope_plan &plan,
                                      const unsigned long long *turns, long long pos, char *row, int d, float scale,
                                      const float (&x0)[8], const float (&x1)[8])
{
    const bool apart = unit.rotated, turned = TURN && apart;
    const float g = fabsf(scale);
    float y[2][8], e[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[0][i] = x0[i];
        y[1][i] = x1[i];
        e[0][i] = e[1][i] = 0.f;
    }
    // element i of chunk k's pair, and whether it is the pair's second
    auto real = [&](int k, int i) {
        const int j = unit.interleaved ? i & ~1 : i;
        const float a = unit.interleaved ? (k ? x1[j] : x0[j]) : x0[j], b = unit.interleaved ? (k ? x1[j + 1] : x0[j + 1]) : x1[j];
        const int pair = unit.interleaved ? ((k ? unit.at1 : unit.at0) + j) / 2 : unit.at0 + j;
        return rotated_real(a, b, unit.interleaved ? i & 1 : k, turns[pair] * (unsigned long long)pos, plan.magnitude);
    };
    if (turned) {
        unit.turn(y[0], y[1]);
        const float f = kRotationError * fabsf(plan.magnitude);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (unit.interleaved) {
                e[0][i] = f * (fabsf(x0[i]) + fabsf(x0[i ^ 1]));
                e[1][i] = f * (fabsf(x1[i]) + fabsf(x1[i ^ 1]));
            } else {
                e[0][i] = e[1][i] = f * (fabsf(x0[i]) + fabsf(x1[i]));
            }
    }
    // magnitudes, what they are known to, NaN of each chunk's block
    float top[2] = {0.f, 0.f}, off[2] = {0.f, 0.f}, nan[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top[k] = fmaxf(top[k], fabsf(y[k][i]));
            off[k] = fmaxf(off[k], e[k][i]);
            nan[k] += y[k][i] * 0.f;  // NaN for an infinity too, which is looked at below
        }
    const unsigned int lane = threadIdx.x & 31, both = 3u << (lane & ~1u);
    if (apart) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            top[k] = fmaxf(top[k], __shfl_xor_sync(both, top[k], 1));
            off[k] = fmaxf(off[k], __shfl_xor_sync(both, off[k], 1));
            nan[k] += __shfl_xor_sync(both, nan[k], 1);
        }
    } else {
        top[0] = top[1] = fmaxf(top[0], top[1]);
        nan[0] = nan[1] = nan[0] + nan[1];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t byte = 0x7fu, codes = 0;
        bool is_nan = nan[k] != 0.f;
        if (is_nan && top[k] == INFINITY) {
            // infinities are saturated unless there is a NaN beside them
            is_nan = false;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                is_nan |= y[k][i] != y[k][i] || (!apart && y[k ^ 1][i] != y[k ^ 1][i]);
            if (apart)
                is_nan |= __shfl_xor_sync(both, (int)is_nan, 1) != 0;
        }
        if (!is_nan) {
            byte = block_scale(top[k], top[k] == INFINITY ? 0.f : off[k], g, [&] {
                double x = 0.0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x = fmax(x, fabs(real(k, i)));
                return fmax(x, __shfl_xor_sync(both, x, 1));  // (both lanes are here: they have the same bounds)
            });
            codes = block_codes(y[k], e[k], e4m3_value(byte), g, [&](int i) { return real(k, i); });
            if (scale < 0.f)
                codes ^= 0x88888888u;
        }
        const int at = k ? unit.at1 : unit.at0;
        *reinterpret_cast<uint32_t *>(row + at / 2) = codes;
        if (at % 16 == 0)
            row[d / 2 + at / 16] = (char)byte;
    }
}

template <int ELEM, int VE, bool FEW>
__global__ void __launch_bounds__(kRotThreads, FEW ? 3 : 2) append_kernel(const __grid_constant__ AppendArgs a)
{
    using T = __nv_bfloat16;
    constexpr bool FP8 = ELEM == MERCURY_ELEM_E4M3, FP4 = ELEM == MERCURY_ELEM_E2M1;
    __shared__ unsigned long long turns[MERCURY_MAX_ROT / 2];
    stage_turns(a.plan, turns);
    chain_wait();
    __syncthreads();
    const int lane_units = kRotThreads / a.tokens_per_block;
    const int group = blockIdx.x % a.head_groups;  // neighbours take the same tokens: their rows adjoin
    const long long token = (long long)(blockIdx.x / (unsigned int)a.head_groups) * a.tokens_per_block + threadIdx.x / lane_units;
    if (token >= a.tokens)
        return;
    const int b = (unsigned int)token / (unsigned int)a.S, i = (int)token - b * a.S;
    const PagedView &c = a.cache;
    const int Hkv = c.Hkv, Hq = a.Hq;
    const int h0 = group * a.heads_per_thread, h1 = min(Hq + 2 * Hkv, h0 + a.heads_per_thread);
    const long long past = a.past[b];
    const int n_new = a.new_lens ? a.new_lens[b] : a.S;
    if ((n_new < 0 || n_new > a.S) && i == 0)
        record_bounds(0x801);
    if (i >= n_new)
        return;
    // the cache row, or none where the position or its page does not exist
    const long long pos = past + i;
    const bool in_table = pos >= 0 && pos < (long long)c.max_pages * c.page_size;
    int page = -1, at = 0;
    if (in_table) {
        at = page_of(c, (int)pos);
        page = c.table[b * c.table_stride + at];
    } else {
        record_bounds(0x802);
    }
    const int row_size = FP4 ? a.d / 2 + a.d / 16 : a.d;  // elements of a row, bytes of a 4-bit one
    const long long head_stride = (long long)c.page_size * row_size;

    for (int u = threadIdx.x % lane_units; u < a.units; u += lane_units) {
        RotUnit<VE> unit(a.plan, u, a.d);
        long long row = -1;  // element offset of head 0's row
        bool known = false;
        auto ready = [&] {
            if (known)
                return;
            known = true;
            if (h0 < Hq + Hkv)
                unit.set_angles(turns, a.plan.magnitude, pos);
            if (page >= 0 && page < c.num_pages)
                row = page * c.page_stride + (pos - (long long)at * c.page_size) * row_size;
            else if (in_table)
                record_bounds(0x803);
        };
        // one head's unit into the cache
        auto keep = [&](char *cache, float scale, int h, const float (&y0)[VE], const float (&y1)[VE]) {
            if (row < 0)
                return;
            const long long to = row + h * head_stride;
            if constexpr (FP8) {
                const Quotient q(scale);
                q.store<VE>((uint8_t *)cache + to + unit.at0, y0);
                if (unit.two)
                    q.store<VE>((uint8_t *)cache + to + unit.at1, y1);
            } else {
                store_chunk<VE>((T *)cache + to + unit.at0, y0);
                if (unit.two)
                    store_chunk<VE>((T *)cache + to + unit.at1, y1);
            }
        };
        // this block's part of the queries, the keys and the values
        const int q1 = min(h1, Hq), k0 = max(h0 - Hq, 0), k1 = min(h1 - Hq, Hkv), v0 = max(h0 - Hq - Hkv, 0),
                  v1 = h1 - Hq - Hkv;
        if (h0 < q1) {
            T *const dst = a.q_out + b * a.os.b + i * a.os.s;
            walk_heads<T, VE, true, false, FEW>(a.q + b * a.qs.b + i * a.qs.s + h0 * a.qs.h, a.qs.h, nullptr, q1 - h0, unit, ready,
                                    [&](int h, const float (&y0)[VE], const float (&y1)[VE], float) {
                                        if (!unit.rotated && !a.copy_rest)
                                            return;
                                        T *p = dst + (h0 + h) * a.os.h;
                                        store_chunk<VE>(p + unit.at0, y0);
                                        if (unit.two)
                                            store_chunk<VE>(p + unit.at1, y1);
                                    });
        }
        if constexpr (FP4) {
            auto keep_row = [&](char *cache, float scale, int h, auto turn, const float (&x0)[VE], const float (&x1)[VE]) {
                if (row >= 0)
                    keep4<decltype(turn)::value>(unit, a.plan, turns, pos, cache + row + h * head_stride, a.d, scale, x0, x1);
            };
            if (k0 < k1)
                walk_heads<T, VE, false, true, FEW>(a.k + b * a.ks.b + i * a.ks.s + k0 * a.ks.h, a.ks.h, c.k_scale + k0, k1 - k0,
                                                    unit, ready, [&](int h, const float (&x0)[VE], const float (&x1)[VE], float scale) {
                                                        keep_row(c.k, scale, k0 + h, Turn<true>(), x0, x1);
                                                    });
            if (v0 < v1)
                walk_heads<T, VE, false, true, FEW>(a.v + b * a.vs.b + i * a.vs.s + v0 * a.vs.h, a.vs.h, c.v_scale + v0, v1 - v0,
                                                    unit, ready, [&](int h, const float (&x0)[VE], const float (&x1)[VE], float scale) {
                                                        keep_row(c.v, scale, v0 + h, Turn<false>(), x0, x1);
                                                    });
            continue;
        }
        if (k0 < k1)
            walk_heads<T, VE, true, FP8, FEW>(a.k + b * a.ks.b + i * a.ks.s + k0 * a.ks.h, a.ks.h,
                                    FP8 ? c.k_scale + k0 : nullptr, k1 - k0, unit, ready,
                                    [&](int h, const float (&y0)[VE], const float (&y1)[VE], float scale) {
                                        keep(c.k, scale, k0 + h, y0, y1);
                                    });
        if (v0 < v1)
            walk_heads<T, VE, false, FP8, FEW>(a.v + b * a.vs.b + i * a.vs.s + v0 * a.vs.h, a.vs.h,
                                     FP8 ? c.v_scale + v0 : nullptr, v1 - v0, unit, ready,
                                     [&](int h, const float (&y0)[VE], const float (&y1)[VE], float scale) {
                                         keep(c.v, scale, v0 + h, y0, y1);
                                     });
    }
}

template <int ELEM, int VE>
int launch(AppendArgs &a, int sms, cudaStream_t stream, char *msg, size_t msg_len)
{
    const RotShape g = rot_shape(a.tokens, a.Hq + 2 * a.cache.Hkv, a.d, a.plan.rot_dim, VE, sms);
    if (g.blocks * g.head_groups > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many tokens for one call (%lld)", (long long)a.tokens);
        return MERCURY_EINVAL;
    }
    a.head_groups = g.head_groups;
    a.units = g.units;
    a.tokens_per_block = g.tokens_per_block;
    a.heads_per_thread = g.heads_per_thread;
    void (*kernel)(AppendArgs) = append_kernel<ELEM, VE, false>;
    if constexpr (VE == 4)
        if (rot_few(g, a.Hq + 2 * a.cache.Hkv, VE, 2, sms))
            kernel = append_kernel<ELEM, VE, true>;
    const cudaError_t e =
        launch_chained(kernel, dim3((unsigned)(g.blocks * g.head_groups)), kRotThreads, 0, stream, a);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache append kernel launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

// Keys and values of any other rotated part or alignment into a 4-bit cache: a
// thread a block of 16 elements of a head, element by element.  (Their queries
// go as with the other caches, by a launch of their own.)
__global__ void __launch_bounds__(kRotThreads) append_blocks_kernel(const __grid_constant__ AppendArgs a)
{
    __shared__ unsigned long long turns[MERCURY_MAX_ROT / 2];
    stage_turns(a.plan, turns);
    chain_wait();
    __syncthreads();
    const PagedView &c = a.cache;
    const int blocks = a.d / 16, heads = 2 * c.Hkv, rot = a.plan.rot_dim, row_size = a.d / 2 + a.d / 16;
    const long long item = (long long)blockIdx.x * kRotThreads + threadIdx.x;
    const long long token = item / (blocks * heads);
    if (token >= a.tokens)
        return;
    const int rest = (int)(item - token * (blocks * heads)), head = rest / blocks, at = rest % blocks * 16;
    const int b = (unsigned int)token / (unsigned int)a.S, i = (int)token - b * a.S;
    const int n_new = a.new_lens ? a.new_lens[b] : a.S;
    if ((n_new < 0 || n_new > a.S) && i == 0 && rest == 0)
        record_bounds(0x801);
    if (i >= n_new)
        return;
    const long long pos = (long long)a.past[b] + i;
    const bool value = head >= c.Hkv;
    const int h = head - (value ? c.Hkv : 0);
    const __nv_bfloat16 *const src = value ? a.v + b * a.vs.b + i * a.vs.s + h * a.vs.h
                                           : a.k + b * a.ks.b + i * a.ks.s + h * a.ks.h;
    // element j's pair, and whether it is its second
    auto pair_of = [&](int j) { return a.plan.interleaved ? j / 2 : j < rot / 2 ? j : j - rot / 2; };
    auto second = [&](int j) { return a.plan.interleaved ? (j & 1) != 0 : j >= rot / 2; };
    auto first_at = [&](int j) { return a.plan.interleaved ? j & ~1 : pair_of(j); };
    const int step = a.plan.interleaved ? 1 : rot / 2;
    float y[16], e[16];
    float top = 0.f, off = 0.f;
    bool nan = false;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int j = at + k;
        e[k] = 0.f;
        if (!value && j < rot) {
            const float x = __bfloat162float(src[first_at(j)]), z = __bfloat162float(src[first_at(j) + step]);
            float cs, sn;
            rope_cos_sin(turns[pair_of(j)], pos, a.plan.magnitude, cs, sn);
            y[k] = second(j) ? z * cs + x * sn : x * cs - z * sn;
            e[k] = kRotationError * fabsf(a.plan.magnitude) * (fabsf(x) + fabsf(z));
        } else {
            y[k] = __bfloat162float(src[j]);
        }
        top = fmaxf(top, fabsf(y[k]));
        off = fmaxf(off, e[k]);
        nan |= y[k] != y[k];
    }
    const bool in_table = pos >= 0 && pos < (long long)c.max_pages * c.page_size;
    if (!in_table) {
        record_bounds(0x802);
        return;
    }
    const int p = page_of(c, (int)pos), page = c.table[b * c.table_stride + p];
    if (page < 0 || page >= c.num_pages) {
        record_bounds(0x803);
        return;
    }
    char *const row = (value ? c.v : c.k) + page * c.page_stride +
                      ((long long)h * c.page_size + pos - (long long)p * c.page_size) * row_size;
    const float scale = (value ? c.v_scale : c.k_scale)[h], g = fabsf(scale);
    auto real = [&](int k) {
        const int j = at + k;
        return rotated_real(__bfloat162float(src[first_at(j)]), __bfloat162float(src[first_at(j) + step]), second(j),
                            turns[pair_of(j)] * (unsigned long long)pos, a.plan.magnitude);
    };
    uint32_t byte = 0x7fu, codes[2] = {0u, 0u};
    if (!nan) {
        byte = block_scale(top, top == INFINITY ? 0.f : off, g, [&] {
            double x = 0.0;
#pragma unroll 1
            for (int k = 0; k < 16; ++k)
                x = fmax(x, at + k < rot && !value ? fabs(real(k)) : fabs((double)__bfloat162float(src[at + k])));
            return x;
        });
        const float s = e4m3_value(byte);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float y8[8], e8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y8[j] = y[8 * k + j];
                e8[j] = e[8 * k + j];
            }
            codes[k] = block_codes(y8, e8, s, g, [&](int j) { return real(8 * k + j); });
            if (scale < 0.f)
                codes[k] ^= 0x88888888u;
        }
    }
    *reinterpret_cast<uint32_t *>(row + at / 2) = codes[0];
    *reinterpret_cast<uint32_t *>(row + at / 2 + 4) = codes[1];
    row[a.d / 2 + at / 16] = (char)byte;
}

int launch_blocks(AppendArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    const long long blocks = (a.tokens * (a.d / 16) * 2 * a.cache.Hkv + kRotThreads - 1) / kRotThreads;
    if (blocks > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many tokens for one call (%lld)", (long long)a.tokens);
        return MERCURY_EINVAL;
    }
    const cudaError_t e = launch_chained(append_blocks_kernel, dim3((unsigned)blocks), kRotThreads, 0, stream, a);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache append kernel launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

}  // namespace

int launch_kv_append(const void *k, const Strides &ks, const void *v, const Strides &vs, const void *q,
                     const Strides &qs, void *q_out, const Strides &os, const mercury_paged_cache &cache,
                     const int *past_lens, const int *new_lens, int B, int Hq, int S, const mercury_rope_plan *plan,
                     int sms, cudaStream_t stream, char *msg, size_t msg_len)
{
    AppendArgs a;
    a.q = (const __nv_bfloat16 *)q;
    a.k = (const __nv_bfloat16 *)k;
    a.v = (const __nv_bfloat16 *)v;
    a.q_out = (__nv_bfloat16 *)q_out;
    a.qs = qs;
    a.ks = ks;
    a.vs = vs;
    a.os = os;
    a.past = past_lens;
    a.new_lens = new_lens;
    a.cache = make_view(cache);
    a.Hq = q ? Hq : 0;
    a.S = S;
    a.d = cache.d;
    a.tokens = (long long)B * S;
    a.copy_rest = !(q == q_out && qs.b == os.b && qs.h == os.h && qs.s == os.s);
    if (plan) {
        a.plan = *plan;
    } else {
        a.plan.rot_dim = 0;
        a.plan.interleaved = 0;
        a.plan.magnitude = 1.f;
    }
    auto fits_q = [&](int VE) {
        return a.plan.rot_dim % (2 * VE) == 0 &&
               (!q || (rot_vector_ok(q, qs, a.d, 2, VE) && rot_vector_ok(q_out, os, a.d, 2, VE)));
    };
    auto fits = [&](int VE) { return fits_q(VE) && rot_vector_ok(k, ks, a.d, 2, VE) && rot_vector_ok(v, vs, a.d, 2, VE); };
    const int VE = fits(8) ? 8 : fits(4) ? 4 : 1;
    constexpr int kBf16 = MERCURY_ELEM_BF16, kE4m3 = MERCURY_ELEM_E4M3, kE2m1 = MERCURY_ELEM_E2M1;
    if (cache.elem == kE2m1) {
        // whole blocks from pairs of lanes: 16-byte accesses, and a rotated part of whole blocks on each side
        if (VE == 8 && a.plan.rot_dim % 32 == 0)
            return launch<kE2m1, 8>(a, sms, stream, msg, msg_len);
        if (q) {
            AppendArgs only = a;
            only.cache.Hkv = 0;
            const int rc = fits_q(8)   ? launch<kBf16, 8>(only, sms, stream, msg, msg_len)
                           : fits_q(4) ? launch<kBf16, 4>(only, sms, stream, msg, msg_len)
                                       : launch<kBf16, 1>(only, sms, stream, msg, msg_len);
            if (rc != MERCURY_OK)
                return rc;
        }
        return launch_blocks(a, stream, msg, msg_len);
    }
    if (cache.elem == kE4m3)
        return VE == 8   ? launch<kE4m3, 8>(a, sms, stream, msg, msg_len)
               : VE == 4 ? launch<kE4m3, 4>(a, sms, stream, msg, msg_len)
                         : launch<kE4m3, 1>(a, sms, stream, msg, msg_len);
    return VE == 8   ? launch<kBf16, 8>(a, sms, stream, msg, msg_len)
           : VE == 4 ? launch<kBf16, 4>(a, sms, stream, msg, msg_len)
                     : launch<kBf16, 1>(a, sms, stream, msg, msg_len);
}

int read_and_clear_append_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    return read_and_clear_words(g_append_err_word, g_append_err_site, "append", word, site, msg, msg_len);
}

}  // namespace mercury
