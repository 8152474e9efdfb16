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
// A 4-bit cache's codes and scales are settled as quantize4.cuh says; a block of
// 16 elements is two lanes' where it lies in the rotated part, and one's else.
//
// Measured on a GB300: a 32K prompt of 32 query and 8 + 8 key and value heads
// of 128, straight from a fused projection: 122 us, 98 % of the measured copy
// bandwidth; one token of 32 sequences: 3.0 us; 6 x 1000 padded tokens of 24
// heads of 64 into an 8-bit cache: 8.2 us, bound by the latency of short
// threads (3 us of bytes).  Into a 4-bit cache: 8K tokens of 32 query and 8 + 8
// key and value heads of 128: 48 us (26 us of bytes), its keys and values alone 28
// us (6 us of bytes; 16 bits 35 and 10 us): not by the quantisation's work (2 us
// of it) but by the little that a thread has on the way, one head, where the
// other caches' have two to four and the next ones.  6 x 1000 padded tokens of 24 heads of 64
// 10.6 us, one token of 32 sequences 3.5 to 4.2 us.  Element by element (other rotated
// parts and alignments): the 8K tokens with 24 elements rotated 87 us, their
// keys and values alone 57; all 128 rotated, heads that begin at odd elements, 122.
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
    int kv_groups, kv_per_thread;  // of a 4-bit cache: those of keys and values, which come first
    long long tokens;
    int copy_rest;  // q_out is not q itself
    mercury_rope_plan plan;
};

// One head's unit (two chunks of 8 elements, as loaded) into a row of a 4-bit
// cache.  The chunks of a unit of the rotated part (turned or, of values, not)
// are halves of two blocks, whose other halves the neighbouring lane has; any
// other unit's make one block.  What has to be settled exactly is settled out of
// line, for it is rare.
template <bool TURN>
__device__ __forceinline__ void keep4(const RotUnit<8> &unit, const mercury_rope_plan &plan,
                                      const unsigned long long *turns, long long pos, char *row, int d, float scale,
                                      const float (&x0)[8], const float (&x1)[8])
{
    const bool apart = unit.rotated, turned = TURN && apart;
    const float g = fabsf(scale);
    float y[2][8], top[2] = {0.f, 0.f}, off[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[0][i] = x0[i];
        y[1][i] = x1[i];
    }
    if (turned) {
        unit.turn(y[0], y[1]);
        float a = 0.f, b = 0.f;  // the largest sum of a pair's magnitudes in each chunk
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a = fmaxf(a, fabsf(x0[i]) + fabsf(unit.interleaved ? x0[i ^ 1] : x1[i]));
            b = fmaxf(b, fabsf(x1[i]) + fabsf(unit.interleaved ? x1[i ^ 1] : x0[i]));
        }
        off[0] = kRotationError * fabsf(plan.magnitude) * a;
        off[1] = kRotationError * fabsf(plan.magnitude) * b;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            top[k] = max_nan(top[k], y[k][i], y[k][i + 1]);
    const unsigned int both = 3u << (threadIdx.x & 30u);
    if (apart) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            top[k] = max_nan(top[k], __shfl_xor_sync(both, top[k], 1));
            if (TURN)
                off[k] = fmaxf(off[k], __shfl_xor_sync(both, off[k], 1));
        }
    } else {
        top[0] = top[1] = max_nan(top[0], top[1]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int at = k ? unit.at1 : unit.at0;
        // an infinity, which is held as 6 * 448, leaves no bounds
        const float by = top[k] < INFINITY ? off[k] : 0.f;
        auto source = [&](float (&first)[8], float (&second)[8], float (&copy)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                copy[i] = y[k][i];
                first[i] = unit.interleaved ? (k ? x1[i & ~1] : x0[i & ~1]) : x0[i];
                second[i] = unit.interleaved ? (k ? x1[i | 1] : x0[i | 1]) : x1[i];
            }
            return Source{first, second, (unsigned long long)pos, turns, plan.magnitude, at, plan.rot_dim, unit.interleaved};
        };
        const uint32_t ends = scale_ends(top[k], by, g);
        uint32_t byte = ends & 0xffu;
        if (byte != ends >> 8) {
            float first[8], second[8], copy[8];
            const Source from = source(first, second, copy);
            byte = settle_scale<8>(byte, ends >> 8, top[k], by, g, copy, by > 0.f ? &from : nullptr, both);
        }
        uint32_t lo, w;
        code_ends(y[k], by, byte == 0x7fu ? 0.f : e4m3_value(byte), g, lo, w);
        if (lo != (w & 0x77777777u)) {
            float first[8], second[8], copy[8];
            const Source from = source(first, second, copy);
            w = settle_codes(lo, w, e4m3_value(byte), g, copy, by > 0.f ? &from : nullptr);
        }
        *reinterpret_cast<uint32_t *>(row + at / 2) = stored_codes(w, scale);
        if (at % 16 == 0)
            row[d / 2 + at / 16] = (char)byte;
    }
}

// The unit of heads h = 0 .. n - 1 into a 4-bit cache: the next head's loads on
// their way while one is turned and stored.
template <bool TURN>
__device__ __forceinline__ void walk4(const __nv_bfloat16 *src, long long stride, const float *scales, int n,
                                      const RotUnit<8> &unit, const mercury_rope_plan &plan,
                                      const unsigned long long *turns, long long pos, char *row, long long head_stride, int d)
{
    Chunk<__nv_bfloat16, 8> a, b;
    float scale = scales[0];
    a.load(src + unit.at0);
    b.load(src + unit.at1);
#pragma unroll 1
    for (int h = 0; h < n; ++h) {
        float x0[8], x1[8];
        a.widen(x0);
        b.widen(x1);
        const float s = scale;
        if (h + 1 < n) {
            a.load(src + (h + 1) * stride + unit.at0);
            b.load(src + (h + 1) * stride + unit.at1);
            scale = scales[h + 1];
        }
        keep4<TURN>(unit, plan, turns, pos, row + h * head_stride, d, s, x0, x1);
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
    int h0 = group * a.heads_per_thread, h1 = min(Hq + 2 * Hkv, h0 + a.heads_per_thread);
    if constexpr (FP4) {
        if (group < a.kv_groups) {
            h0 = Hq + group * a.kv_per_thread;
            h1 = min(Hq + 2 * Hkv, h0 + a.kv_per_thread);
        } else {
            h0 = (group - a.kv_groups) * a.heads_per_thread;
            h1 = min(Hq, h0 + a.heads_per_thread);
        }
    }
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
            ready();
            if (k0 < k1 && row >= 0)
                walk4<true>(a.k + b * a.ks.b + i * a.ks.s + k0 * a.ks.h, a.ks.h, c.k_scale + k0, k1 - k0, unit, a.plan, turns,
                            pos, c.k + row + k0 * head_stride, head_stride, a.d);
            if (v0 < v1 && row >= 0)
                walk4<false>(a.v + b * a.vs.b + i * a.vs.s + v0 * a.vs.h, a.vs.h, c.v_scale + v0, v1 - v0, unit, a.plan, turns,
                             pos, c.v + row + v0 * head_stride, head_stride, a.d);
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
    RotShape g = rot_shape(a.tokens, a.Hq + 2 * a.cache.Hkv, a.d, a.plan.rot_dim, VE, sms);
    if constexpr (ELEM == MERCURY_ELEM_E2M1) {
        // A 4-bit key or value takes a thread several times as long as a query
        // does: they go by fewer heads a thread, and first (8K tokens of 32 + 8 +
        // 8 heads, and 32K read back: 75.1 us, with one rule for all 80.4).
        const RotShape q = rot_shape(a.tokens, a.Hq > 0 ? a.Hq : 1, a.d, a.plan.rot_dim, VE, sms);
        const int kv = 2 * a.cache.Hkv;
        int most = 4;
        while (most > 1 && g.blocks * ((kv + most - 1) / most) < 2LL * sms)
            most /= 2;
        a.kv_per_thread = most;
        a.kv_groups = (kv + most - 1) / most;
        g.heads_per_thread = q.heads_per_thread;
        g.head_groups = a.kv_groups + (a.Hq + q.heads_per_thread - 1) / q.heads_per_thread;
    }
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
    float y[16], x[16], z[16];
    float top = 0.f, off = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int j = at + k;
        if (!value && j < rot) {
            x[k] = __bfloat162float(src[first_at(j)]);
            z[k] = __bfloat162float(src[first_at(j) + step]);
            float cs, sn;
            rope_cos_sin(turns[pair_of(j)], pos, a.plan.magnitude, cs, sn);
            y[k] = second(j) ? z[k] * cs + x[k] * sn : x[k] * cs - z[k] * sn;
            off = fmaxf(off, kRotationError * fabsf(a.plan.magnitude) * (fabsf(x[k]) + fabsf(z[k])));
        } else {
            // (of itself and no partner at no angle, where a block's part is turned)
            x[k] = z[k] = y[k] = __bfloat162float(src[j]);
        }
        top = max_nan(top, y[k]);
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
    const float by = top < INFINITY ? off : 0.f;
    Source from = {x, z, (unsigned long long)pos, turns, a.plan.magnitude, at, rot, a.plan.interleaved};
    const uint32_t ends = scale_ends(top, by, g);
    uint32_t byte = ends & 0xffu;
    if (byte != ends >> 8)
        byte = settle_scale<16>(byte, ends >> 8, top, by, g, y, by > 0.f ? &from : nullptr, 0u);
    const float s = byte == 0x7fu ? 0.f : e4m3_value(byte);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float part[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            part[j] = y[8 * k + j];
        uint32_t lo, w;
        code_ends(part, by, s, g, lo, w);
        if (lo != (w & 0x77777777u)) {
            const Source half = {x + 8 * k, z + 8 * k, from.pos, turns, a.plan.magnitude, at + 8 * k, rot, a.plan.interleaved};
            w = settle_codes(lo, w, s, g, y + 8 * k, by > 0.f ? &half : nullptr);
        }
        *reinterpret_cast<uint32_t *>(row + at / 2 + 4 * k) = stored_codes(w, scale);
    }
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
