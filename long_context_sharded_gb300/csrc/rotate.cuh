// rotate.cuh -- the work split and the element arithmetic that the rotation
// and the cache append share.
//
// A head of d elements is cut into column units of VE-element chunks (16 bytes;
// 8 bytes for 16-bit elements whose rotated part is a multiple of 8 but not of
// 16, or whose strides are of 8 bytes; else VE = 1).  The
// first rot/(2 VE) units hold two chunks of the rotated part each, j and
// j + rot/(2 VE): with half-split pairs these are the two sides of the same VE
// pairs, with interleaved ones two times VE/2 whole pairs, so both layouts
// read and write the same way and differ only in which registers meet.  The
// rest of the head follows as units of two plain chunks.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "paged.cuh"

namespace mercury {

constexpr int kRotThreads = 256;
constexpr int kRotBatch = 4;  // heads that a thread loads at a time

template <typename T, int VE>
struct Chunk;

template <>
struct Chunk<__nv_bfloat16, 8> {
    uint4 w = {0, 0, 0, 0};
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void widen(float (&y)[8]) const
    {
        y[0] = bf16_lo(w.x), y[1] = bf16_hi(w.x), y[2] = bf16_lo(w.y), y[3] = bf16_hi(w.y);
        y[4] = bf16_lo(w.z), y[5] = bf16_hi(w.z), y[6] = bf16_lo(w.w), y[7] = bf16_hi(w.w);
    }
};

template <>
struct Chunk<__nv_bfloat16, 4> {
    uint2 w = {0, 0};
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void widen(float (&y)[4]) const
    {
        y[0] = bf16_lo(w.x), y[1] = bf16_hi(w.x), y[2] = bf16_lo(w.y), y[3] = bf16_hi(w.y);
    }
};

template <>
struct Chunk<__nv_bfloat16, 1> {
    __nv_bfloat16 w = __nv_bfloat16();
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *p; }
    __device__ __forceinline__ void widen(float (&y)[1]) const { y[0] = __bfloat162float(w); }
};

template <>
struct Chunk<float, 4> {
    float4 w = {0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void load(const float *p) { w = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void widen(float (&y)[4]) const { y[0] = w.x, y[1] = w.y, y[2] = w.z, y[3] = w.w; }
};

template <>
struct Chunk<float, 1> {
    float w = 0.f;
    __device__ __forceinline__ void load(const float *p) { w = *p; }
    __device__ __forceinline__ void widen(float (&y)[1]) const { y[0] = w; }
};

// Each result is rounded once, from its 32-bit value, to the output's type.
template <int VE>
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *p, const float (&y)[VE])
{
    if constexpr (VE == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                   pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    else if constexpr (VE == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    else
        *p = __float2bfloat16_rn(y[0]);
}

template <int VE>
__device__ __forceinline__ void store_chunk(float *p, const float (&y)[VE])
{
    if constexpr (VE == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(y[0], y[1], y[2], y[3]);
    else
        *p = y[0];
}

// y / scale[head] to the nearest e4m3 and saturated.  The stored byte is the one
// nearest to the quotient's 32-bit rounding, as a division gives it, mostly
// without dividing: with r the rounded reciprocal, y r (1 -+ 2^-21) lie on the
// two sides of that quotient (four roundings of 2^-24 each do not reach 2^-21),
// so where both round to the same byte it is the quotient's.  Where they do not
// (next to a tie), or r is zero, infinite or near either, the elements are
// divided.  (6 x 1000 tokens of 24 heads of 64: 10.6 us with divisions
// throughout, 8.2 so; 6 x 8000 of 48 heads of 128: 138 and 122.)
struct Quotient {
    float scale, lo, hi;
    bool divide;

    __device__ __forceinline__ explicit Quotient(float s) : scale(s)
    {
        const float r = 1.f / s;
        lo = r * (1.f - 0x1p-21f);
        hi = r * (1.f + 0x1p-21f);
        divide = !(fabsf(r) > 0x1p-100f && fabsf(r) < 0x1p100f);
    }

    template <int VE>
    __device__ __forceinline__ void store(uint8_t *p, const float (&y)[VE]) const
    {
        constexpr int N = VE == 1 ? 1 : VE / 2;
        uint32_t w[N], differ = divide;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float a = y[2 * i], b = VE == 1 ? 0.f : y[2 * i + (VE > 1)];
            w[i] = pack_e4m3(a * lo, b * lo);
            differ |= w[i] ^ pack_e4m3(a * hi, b * hi);
        }
        if (differ) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = pack_e4m3(y[2 * i] / scale, VE == 1 ? 0.f : y[2 * i + (VE > 1)] / scale);
        }
        if constexpr (VE == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        else if constexpr (VE == 4)
            *reinterpret_cast<uint32_t *>(p) = w[0] | w[1] << 16;
        else
            *p = (uint8_t)w[0];
    }
};

// The plan's frequencies into shared memory: lanes want different ones, which
// the parameter bank would serve one after the other, for every warp anew.
// They are no other kernel's work, so this goes before chain_wait.
__device__ __forceinline__ void stage_turns(const mercury_rope_plan &plan, unsigned long long *turns)
{
    for (int i = threadIdx.x; i < plan.rot_dim / 2; i += kRotThreads)
        turns[i] = plan.turns[i];
}

// One column unit at one position: where its chunks lie, and its rotation.
template <int VE>
struct RotUnit {
    int at0, at1;   // first element of each chunk
    bool two;       // the second chunk exists
    bool rotated;
    bool interleaved;
    float c[VE], s[VE];

    __device__ __forceinline__ RotUnit(const mercury_rope_plan &plan, int u, int d)
    {
        const int rot = plan.rot_dim, n = rot / (2 * VE);
        interleaved = plan.interleaved != 0;
        rotated = u < n;
        two = true;
        if (!rotated) {
            at0 = rot + (u - n) * 2 * VE;
            at1 = at0 + VE;
            two = at1 < d;
        } else if (VE == 1 && interleaved) {
            at0 = 2 * u;
            at1 = at0 + 1;
        } else {
            at0 = u * VE;
            at1 = at0 + rot / 2;
        }
    }

    // turns: the plan's, in shared memory
    __device__ __forceinline__ void set_angles(const unsigned long long *turns, float magnitude, long long pos)
    {
        if (!rotated)
            return;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            // pair of slot i: chunk element i, or for interleaved chunks
            // pairs at0/2 + i (first chunk) and at1/2 + i - VE/2 (second)
            int pair = at0 + i;
            if (interleaved)
                pair = VE == 1 ? at0 / 2 : (i < VE / 2 ? at0 / 2 + i : at1 / 2 + i - VE / 2);
            rope_cos_sin(turns[pair], pos, magnitude, c[i], s[i]);
        }
    }

    __device__ __forceinline__ void turn(float (&y0)[VE], float (&y1)[VE]) const
    {
        if (!rotated)
            return;
        if (VE > 1 && interleaved) {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                const float a = y0[2 * i], b = y0[2 * i + 1], e = y1[2 * i], f = y1[2 * i + 1];
                y0[2 * i] = a * c[i] - b * s[i];
                y0[2 * i + 1] = b * c[i] + a * s[i];
                y1[2 * i] = e * c[i + VE / 2] - f * s[i + VE / 2];
                y1[2 * i + 1] = f * c[i + VE / 2] + e * s[i + VE / 2];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float a = y0[i], b = y1[i];
                y0[i] = a * c[i] - b * s[i];
                y1[i] = b * c[i] + a * s[i];
            }
        }
    }
};

// One unit of n heads, `stride` elements apart from `src` on: turned if TURN,
// and given to store(head, chunk 0, chunk 1, scale).  kRotBatch heads are
// loaded at a time, the first ones while ready(), which has the angles and
// whatever a store needs found, runs.  16-bit heads are double buffered, the next batch on
// its way while one is turned and stored (32K prompt of 40 heads: 109 to 99
// us); 32-bit ones are not: with twice the bytes in flight a head the registers
// cost more than the overlap gains (12.0 against 10.9 us at 2 x 12 heads x
// 4099 tokens).  (Written out, because the output may be the input: the
// compiler would keep each load behind the stores before it.)  With SCALED,
// scales[head] goes the same way; two heads at a time then, since with the
// quantisation's registers four spill (6 x 1000 tokens of 24 heads of 64: 8.2
// us instead of 10.8; 6 x 8000 of 48 of 128: 122 and 150).  Twice as many of
// 8-byte chunks, for as many bytes on the way (32K prompt of 40 heads, 24
// elements rotated: 118 us instead of 134).  FEW: see rot_few.
template <typename T, int VE, bool TURN, bool SCALED, bool FEW, typename Ready, typename Store>
__device__ __forceinline__ void walk_heads(const T *src, long long stride, const float *scales, int n,
                                           RotUnit<VE> &unit, Ready ready, Store store)
{
    constexpr bool kAhead = sizeof(T) == 2 && !FEW;
    constexpr int kBatch = (SCALED ? kRotBatch / 2 : kRotBatch) * (VE * sizeof(T) == 8 && !FEW ? 2 : 1);
    Chunk<T, VE> x0[2][kBatch], x1[2][kBatch];
    float sc[2][kBatch];
    auto load = [&](int slot, int h0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (h0 + i < n) {
                const T *p = src + (h0 + i) * stride;
                x0[slot][i].load(p + unit.at0);
                if (unit.two)
                    x1[slot][i].load(p + unit.at1);
                if constexpr (SCALED)
                    sc[slot][i] = scales[h0 + i];
            }
    };
    load(0, 0);
    ready();
    for (int h0 = 0; h0 < n; h0 += kBatch) {
        if (kAhead)
            load(1, h0 + kBatch);
        else if (h0 > 0)
            load(0, h0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (h0 + i < n) {
                float y0[VE], y1[VE];
                x0[0][i].widen(y0);
                x1[0][i].widen(y1);
                if (TURN)
                    unit.turn(y0, y1);
                if constexpr (SCALED)
                    store(h0 + i, y0, y1, sc[0][i]);
                else
                    store(h0 + i, y0, y1, 1.f);
            }
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                x0[0][i] = x0[1][i];
                x1[0][i] = x1[1][i];
                if constexpr (SCALED)
                    sc[0][i] = sc[1][i];
            }
        }
    }
}

// Grid of a launch over `tokens` tokens of H heads.
struct RotShape {
    int units, tokens_per_block, heads_per_thread, head_groups;
    long long blocks;
};

inline RotShape rot_shape(long long tokens, int H, int d, int rot, int VE, int sms)
{
    RotShape g;
    g.units = rot / (2 * VE) + (d - rot + 2 * VE - 1) / (2 * VE);
    int lanes = 1;  // threads along a token's units: a power of two
    while (lanes < g.units && lanes < kRotThreads)
        lanes *= 2;
    g.tokens_per_block = kRotThreads / lanes;
    g.blocks = (tokens + g.tokens_per_block - 1) / g.tokens_per_block;
    // Heads per thread: as many as leave three blocks for two SMs, at most 16.
    // An angle costs about as much as moving two heads, so a thread of many
    // heads is cheap (a 32K prompt of 40 heads: 138 us with 4, 113 with 8, 99
    // with 16, 102 with 32), but a short call needs its blocks (6 x 1000
    // tokens of 24 heads into an 8-bit cache, with a division for every element: 12.8 us with 16,
    // 11.7 with 2).
    int hp = 16;
    while (hp > 1 && 2 * g.blocks * ((H + hp - 1) / hp) < 3LL * sms)
        hp /= 2;
    g.heads_per_thread = hp;
    g.head_groups = (H + hp - 1) / hp;
    return g;
}

// Whether a call takes the variant for a token's few heads, where a thread's
// life is one batch: nothing loaded ahead, and the registers that frees spent
// on a third block an SM.  (8-byte chunks, 24 elements rotated: 10 x 15475
// tokens of 3 heads of 128 into a cache 61 us instead of 96, 32K of 2 heads
// rotated 13.4 instead of 19.5; up to two blocks an SM there is no third, and
// with 16-byte chunks it would spill: 3 heads 15.9 instead of 15.5.)
inline bool rot_few(const RotShape &g, int H, int VE, int elem_size, int sms)
{
    return VE * elem_size == 8 && H <= kRotBatch && g.blocks * g.head_groups > 2LL * sms;
}

// Whether every chunk of VE elements of a tensor with these strides starts on
// a multiple of its bytes.
inline bool rot_vector_ok(const void *p, const Strides &s, int d, int elem_size, int VE)
{
    return (uintptr_t)p % (VE * elem_size) == 0 && d % VE == 0 && s.b % VE == 0 && s.h % VE == 0 && s.s % VE == 0;
}

}  // namespace mercury
