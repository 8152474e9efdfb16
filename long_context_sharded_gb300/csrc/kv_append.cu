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
// three tensors, and position, page and angles are found once per thread.
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
    int Hq, S, d, heads_per_thread, units, tokens_per_block;
    long long tokens;
    int copy_rest;  // q_out is not q itself
    mercury_rope_plan plan;
};

template <bool FP8, int VE>
__global__ void __launch_bounds__(kRotThreads) append_kernel(const __grid_constant__ AppendArgs a)
{
    using T = __nv_bfloat16;
    chain_wait();
    const int lane_units = kRotThreads / a.tokens_per_block;
    const long long token = (long long)blockIdx.x * a.tokens_per_block + threadIdx.x / lane_units;
    if (token >= a.tokens)
        return;
    const int b = (int)(token / a.S), i = (int)(token % a.S);
    int n_new = a.S;
    if (a.new_lens) {
        n_new = a.new_lens[b];
        if ((n_new < 0 || n_new > a.S) && i == 0)
            record_bounds(0x801);
    }
    if (i >= n_new)
        return;
    const PagedView &c = a.cache;
    const int Hkv = c.Hkv, Hq = a.Hq;
    const int h0 = blockIdx.y * a.heads_per_thread, h1 = min(Hq + 2 * Hkv, h0 + a.heads_per_thread);

    // the cache row, or none where the position or its page does not exist
    const long long pos = (long long)a.past[b] + i;
    long long row = -1;  // element offset of head 0's row
    if (pos < 0 || pos >= (long long)c.max_pages * c.page_size) {
        record_bounds(0x802);
    } else {
        const int at = page_of(c, (int)pos);
        const int page = c.table[b * c.table_stride + at];
        if (page < 0 || page >= c.num_pages)
            record_bounds(0x803);
        else
            row = page * c.page_stride + (pos - (long long)at * c.page_size) * a.d;
    }
    const long long head_stride = (long long)c.page_size * a.d;

    for (int u = threadIdx.x % lane_units; u < a.units; u += lane_units) {
        const RotUnit<VE> unit(a.plan, u, a.d, pos, false);
        for (int hb = h0; hb < h1; hb += kRotBatch) {
            Chunk<T, VE> x0[kRotBatch], x1[kRotBatch];
#pragma unroll
            for (int j = 0; j < kRotBatch; ++j) {
                const int h = hb + j;
                if (h < h1) {
                    const T *p = h < Hq         ? a.q + b * a.qs.b + i * a.qs.s + h * a.qs.h
                                 : h < Hq + Hkv ? a.k + b * a.ks.b + i * a.ks.s + (h - Hq) * a.ks.h
                                                : a.v + b * a.vs.b + i * a.vs.s + (h - Hq - Hkv) * a.vs.h;
                    x0[j].load(p + unit.at0);
                    if (unit.two)
                        x1[j].load(p + unit.at1);
                }
            }
#pragma unroll
            for (int j = 0; j < kRotBatch; ++j) {
                const int h = hb + j;
                if (h >= h1)
                    continue;
                float y0[VE], y1[VE];
                x0[j].widen(y0);
                x1[j].widen(y1);
                if (h < Hq + Hkv)
                    unit.turn(y0, y1);
                if (h < Hq) {
                    T *p = a.q_out + b * a.os.b + i * a.os.s + h * a.os.h;
                    if (unit.rotated || a.copy_rest) {
                        store_chunk<VE>(p + unit.at0, y0);
                        if (unit.two)
                            store_chunk<VE>(p + unit.at1, y1);
                    }
                    continue;
                }
                if (row < 0)
                    continue;
                const bool is_k = h < Hq + Hkv;
                const int hk = is_k ? h - Hq : h - Hq - Hkv;
                const long long at = row + hk * head_stride;
                if constexpr (FP8) {
                    // divided, not multiplied by a reciprocal: the stored
                    // byte is the nearest one to the exact quotient's 32-bit
                    // rounding
                    const float sc = (is_k ? c.k_scale : c.v_scale)[hk];
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        y0[e] = y0[e] / sc;
                        y1[e] = y1[e] / sc;
                    }
                    uint8_t *p = (uint8_t *)(is_k ? c.k : c.v) + at;
                    store_chunk_e4m3<VE>(p + unit.at0, y0);
                    if (unit.two)
                        store_chunk_e4m3<VE>(p + unit.at1, y1);
                } else {
                    T *p = (T *)(is_k ? c.k : c.v) + at;
                    store_chunk<VE>(p + unit.at0, y0);
                    if (unit.two)
                        store_chunk<VE>(p + unit.at1, y1);
                }
            }
        }
    }
}

template <bool FP8, int VE>
int launch(AppendArgs &a, int sms, cudaStream_t stream, char *msg, size_t msg_len)
{
    const RotShape g = rot_shape(a.tokens, a.Hq + 2 * a.cache.Hkv, a.d, a.plan.rot_dim, VE, sms);
    a.units = g.units;
    a.tokens_per_block = g.tokens_per_block;
    a.heads_per_thread = g.heads_per_thread;
    const cudaError_t e = launch_chained(append_kernel<FP8, VE>, dim3((unsigned)g.blocks, (unsigned)g.head_groups),
                                         kRotThreads, 0, stream, a);
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
    const bool wide = rot_vector_ok(k, ks, a.d, 2) && rot_vector_ok(v, vs, a.d, 2) && a.plan.rot_dim % 16 == 0 &&
                      (!q || (rot_vector_ok(q, qs, a.d, 2) && rot_vector_ok(q_out, os, a.d, 2)));
    if (cache.elem == MERCURY_ELEM_E4M3)
        return wide ? launch<true, 8>(a, sms, stream, msg, msg_len) : launch<true, 1>(a, sms, stream, msg, msg_len);
    return wide ? launch<false, 8>(a, sms, stream, msg, msg_len) : launch<false, 1>(a, sms, stream, msg, msg_len);
}

int read_and_clear_append_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    unsigned int zero = 0, w = 0, st = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_append_err_word, sizeof w);
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbol(&st, g_append_err_site, sizeof st);
    if (e == cudaSuccess && (w || st)) {
        e = cudaMemcpyToSymbol(g_append_err_word, &zero, sizeof zero);
        if (e == cudaSuccess)
            e = cudaMemcpyToSymbol(g_append_err_site, &zero, sizeof zero);
    }
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "reading the append error word: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    *word = w;
    *site = st;
    return MERCURY_OK;
}

}  // namespace mercury
