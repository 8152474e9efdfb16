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

template <bool FP8, int VE, bool FEW>
__global__ void __launch_bounds__(kRotThreads, FEW ? 3 : 2) append_kernel(const __grid_constant__ AppendArgs a)
{
    using T = __nv_bfloat16;
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
    const long long head_stride = (long long)c.page_size * a.d;

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
                row = page * c.page_stride + (pos - (long long)at * c.page_size) * a.d;
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

template <bool FP8, int VE>
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
    void (*kernel)(AppendArgs) = append_kernel<FP8, VE, false>;
    if constexpr (VE == 4)
        if (rot_few(g, a.Hq + 2 * a.cache.Hkv, VE, 2, sms))
            kernel = append_kernel<FP8, VE, true>;
    const cudaError_t e =
        launch_chained(kernel, dim3((unsigned)(g.blocks * g.head_groups)), kRotThreads, 0, stream, a);
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
    auto fits = [&](int VE) {
        return rot_vector_ok(k, ks, a.d, 2, VE) && rot_vector_ok(v, vs, a.d, 2, VE) && a.plan.rot_dim % (2 * VE) == 0 &&
               (!q || (rot_vector_ok(q, qs, a.d, 2, VE) && rot_vector_ok(q_out, os, a.d, 2, VE)));
    };
    const int VE = fits(8) ? 8 : fits(4) ? 4 : 1;
    if (cache.elem == MERCURY_ELEM_E4M3)
        return VE == 8   ? launch<true, 8>(a, sms, stream, msg, msg_len)
               : VE == 4 ? launch<true, 4>(a, sms, stream, msg, msg_len)
                         : launch<true, 1>(a, sms, stream, msg, msg_len);
    return VE == 8   ? launch<false, 8>(a, sms, stream, msg, msg_len)
           : VE == 4 ? launch<false, 4>(a, sms, stream, msg, msg_len)
                     : launch<false, 1>(a, sms, stream, msg, msg_len);
}

int read_and_clear_append_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    return read_and_clear_words(g_append_err_word, g_append_err_site, "append", word, site, msg, msg_len);
}

}  // namespace mercury
