// rope.cu -- rotary positions: the plan's frequencies (host) and the rotation
// of every head of a prompt or of single tokens.
//
// For pair i of a head at position p, with angle t = p * f_i and magnitude m,
//     (a, b) -> m (a cos t - b sin t, b cos t + a sin t),
// and with the angle negated for the transpose, which carries gradients back.
// A pair is (i, i + rot/2) or (2i, 2i + 1); the elements from rot on pass
// unchanged.
//
// Memory bound: every element is read and written once, three multiply-adds a
// pair.  A thread owns one column unit of one token (two 16-byte chunks: the
// two halves of the same pairs, or two chunks of whole pairs) and keeps the
// unit's cosines and sines in registers while it walks over the token's
// heads, so an angle is computed once per token and group of heads, not once
// per head.
//
// Measured on a GB300: 40 heads of 128 of a 32K prompt, from a fused
// projection: 99 us, the measured copy bandwidth; 2 x 12 heads of 64 x 4099
// tokens in 32 bits: 10.2 us, 73 %, of which 2 are the launch; one token of 8
// sequences: 2.1 us.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "rotate.cuh"

namespace mercury {

namespace {

struct RopeArgs {
    const void *x;
    void *out;
    const int *pos;
    Strides xs, os;
    long long start, pos_stride;
    int heads_adjoin, blocks, H, S, d, head_groups, heads_per_thread, units, tokens_per_block;
    long long tokens;
    int inverse, copy_rest;
    mercury_rope_plan plan;
};

template <typename T, int VE, bool FEW>
__global__ void __launch_bounds__(kRotThreads, FEW ? 3 : 2) rope_kernel(const __grid_constant__ RopeArgs a)
{
    __shared__ unsigned long long turns[MERCURY_MAX_ROT / 2];
    stage_turns(a.plan, turns);
    chain_wait();
    __syncthreads();
    const int lane_units = kRotThreads / a.tokens_per_block;
    // neighbouring blocks take what adjoins in memory: the next heads of the
    // same tokens, or the next tokens of the same heads
    const int group = a.heads_adjoin ? blockIdx.x % (unsigned int)a.head_groups : blockIdx.x / (unsigned int)a.blocks;
    const long long token = (long long)(a.heads_adjoin ? blockIdx.x / (unsigned int)a.head_groups
                                                       : blockIdx.x - (unsigned int)group * a.blocks) * a.tokens_per_block +
                            threadIdx.x / lane_units;
    if (token >= a.tokens)
        return;
    const int b = (unsigned int)token / (unsigned int)a.S, s = (int)token - b * a.S;
    const int h0 = group * a.heads_per_thread, h1 = min(a.H, h0 + a.heads_per_thread);
    const T *src = (const T *)a.x + b * a.xs.b + s * a.xs.s;
    T *dst = (T *)a.out + b * a.os.b + s * a.os.s;
    for (int u = threadIdx.x % lane_units; u < a.units; u += lane_units) {
        RotUnit<VE> unit(a.plan, u, a.d);
        if (!unit.rotated && !a.copy_rest)
            continue;
        walk_heads<T, VE, true, false, FEW>(
            src + h0 * a.xs.h, a.xs.h, nullptr, h1 - h0, unit,
            [&] {
                const long long pos = a.pos ? a.pos[b * a.pos_stride + s] : a.start + s;
                unit.set_angles(turns, a.plan.magnitude, a.inverse ? -pos : pos);
            },
            [&](int h, const float (&y0)[VE], const float (&y1)[VE], float) {
                T *p = dst + (h0 + h) * a.os.h;
                store_chunk<VE>(p + unit.at0, y0);
                if (unit.two)
                    store_chunk<VE>(p + unit.at1, y1);
            });
    }
}

template <typename T, int VE>
int launch(RopeArgs &a, int B, int sms, cudaStream_t stream, char *msg, size_t msg_len)
{
    const RotShape g = rot_shape(a.tokens, a.H, a.d, a.plan.rot_dim, VE, sms);
    if (g.blocks * g.head_groups > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many tokens for one call (%lld)", (long long)a.tokens);
        return MERCURY_EINVAL;
    }
    a.head_groups = g.head_groups;
    a.blocks = (int)g.blocks;
    a.heads_adjoin = a.xs.h < a.xs.s;
    a.units = g.units;
    a.tokens_per_block = g.tokens_per_block;
    a.heads_per_thread = g.heads_per_thread;
    void (*kernel)(RopeArgs) = rope_kernel<T, VE, false>;
    if constexpr (VE * sizeof(T) == 8)
        if (rot_few(g, a.H, VE, sizeof(T), sms))
            kernel = rope_kernel<T, VE, true>;
    const cudaError_t e =
        launch_chained(kernel, dim3((unsigned)(g.blocks * g.head_groups)), kRotThreads, 0, stream, a);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "rope kernel launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

}  // namespace

int launch_rope(const void *x, const Strides &xs, const int *pos, long long pos_stride, long long start, int B, int H,
                int S, int d, int elem, const mercury_rope_plan &plan, int inverse, void *out, const Strides &os,
                int sms, cudaStream_t stream, char *msg, size_t msg_len)
{
    RopeArgs a;
    a.x = x;
    a.out = out;
    a.pos = pos;
    a.xs = xs;
    a.os = os;
    a.start = start;
    a.pos_stride = pos_stride;
    a.H = H;
    a.S = S;
    a.d = d;
    a.tokens = (long long)B * S;
    a.inverse = inverse;
    // in place, the elements behind the rotated ones are where they belong
    a.copy_rest = !(x == out && xs.b == os.b && xs.h == os.h && xs.s == os.s);
    a.plan = plan;
    const int es = elem == MERCURY_ELEM_FP32 ? 4 : 2;
    auto fits = [&](int VE) {
        return rot_vector_ok(x, xs, d, es, VE) && rot_vector_ok(out, os, d, es, VE) && plan.rot_dim % (2 * VE) == 0;
    };
    if (elem == MERCURY_ELEM_FP32)
        return fits(4) ? launch<float, 4>(a, B, sms, stream, msg, msg_len)
                       : launch<float, 1>(a, B, sms, stream, msg, msg_len);
    return fits(8)   ? launch<__nv_bfloat16, 8>(a, B, sms, stream, msg, msg_len)
           : fits(4) ? launch<__nv_bfloat16, 4>(a, B, sms, stream, msg, msg_len)
                     : launch<__nv_bfloat16, 1>(a, B, sms, stream, msg, msg_len);
}

}  // namespace mercury
