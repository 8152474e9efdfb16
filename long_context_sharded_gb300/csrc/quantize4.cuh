// quantize4.cuh -- blocks of 16 elements as e2m1 codes under an e4m3 scale.
//
// With g the head's scale, a block's scale is s = the e4m3 nearest to its
// largest magnitude over 6 |g|, and an element's code the e2m1 nearest to x /
// (s g), ties to even both times, of the real values: an element that was
// rotated is taken as its rotation is, not as 32 bits round it, so that what a
// cache holds does not hang on how sines are computed or sums are ordered.
//
// A value known to e (0 where it was not rotated) has its quotient bracketed by
// two 32-bit products, wider by 2^-21 than e, which covers their roundings (four
// of 2^-24); where both ends round to the same code, that is it.  Where they do
// not, the border between the two is next to the value, and the two are
// compared: exactly in 32 bits, by the product's rounding error, or for a
// rotated value in 64 bits (one in some 10^5; as 0.2 % of warps meet one, that
// costs little).
#pragma once
#include <stdint.h>

#include "paged.cuh"

namespace mercury {

// Two floats as the nearest e2m1 codes (saturated at 6), lo in the lower half
// of the byte.
__device__ __forceinline__ uint32_t pack_e2m1(float lo, float hi)
{
    uint16_t r;
    asm("{\n\t.reg .b8 x;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %1, %2;\n\tmov.b16 %0, {x, 0};\n\t}" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    const uint32_t w = e4m3_to_f16(byte);
    return __half2float(__ushort_as_half((unsigned short)w));
}

// The sign of x - m g, exactly: x lies next to m g, and m has few bits.
__device__ __forceinline__ int side_of(float x, float m, float g)
{
    const float p = __fmul_rn(m, g), d = __fsub_rn(x, p), e = __fmaf_rn(m, g, -p);
    return d > e ? 1 : d < e ? -1 : 0;
}

__device__ __forceinline__ int side_of(double x, float m, float g)
{
    const double p = (double)m * g;
    return x > p ? 1 : x < p ? -1 : 0;
}

constexpr float kWider = 0x1p-21f;

// What a block's elements are known to: a rotated element (a c - b s) of 32-bit
// sine and cosine is off by at most this times |a| + |b| (the angle's rounding
// 9.4e-8, and five roundings of 6e-8 each).
constexpr float kRotationError = 6e-7f;

// The scale's byte.  amax: the largest magnitude, known to e; g > 0;
// real(): the largest magnitude in 64 bits, asked for where e > 0.
template <typename Real>
__device__ __forceinline__ uint32_t block_scale(float amax, float e, float g, Real real)
{
    if (amax == INFINITY)
        return 0x7eu;
    const float r = 1.f / (6.f * g);
    const uint32_t both = pack_e4m3(fmaxf(amax - e, 0.f) * r * (1.f - kWider), (amax + e) * r * (1.f + kWider));
    const uint32_t lo = both & 0xffu, hi = both >> 8;
    if (lo == hi)
        return lo;
    const float m = 3.f * (e4m3_value(lo) + e4m3_value(hi));  // 6 times the border between them
    const int side = e > 0.f ? side_of(real(), m, g) : side_of(amax, m, g);
    return side > 0 || (side == 0 && (lo & 1u)) ? hi : lo;
}

// N codes, four bits each.  y: the elements, known to e[]; s, g > 0: the scales;
// real(i): element i in 64 bits, asked for where e[i] > 0.
template <int N, typename Real>
__device__ __forceinline__ uint32_t block_codes(const float (&y)[N], const float (&e)[N], float s, float g, Real real)
{
    uint32_t w = 0, differ = 0;
    // where s is zero the codes are, and where s g has left the 32-bit range the
    // codes are what the products make of that
    const float r = s > 0.f ? 1.f / (s * g) : 0.f;
    const float below = r * (1.f - kWider), above = r * (1.f + kWider);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float a = fabsf(y[i]), b = fabsf(y[i + 1]);
        const uint32_t lo = pack_e2m1(fmaxf(a - e[i], 0.f) * below, fmaxf(b - e[i + 1], 0.f) * below);
        const uint32_t hi = pack_e2m1((a + e[i]) * above, (b + e[i + 1]) * above);
        w |= lo << (4 * i);
        differ |= (lo ^ hi) << (4 * i);
    }
    if (differ) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (differ >> (4 * i) & 15u) {
                const uint32_t c = w >> (4 * i) & 7u;
                // the border above code c: 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5
                const float m = s * (c < 4 ? 0.5f * c + 0.25f : c < 6 ? (float)c - 1.5f : 5.f);
                const int side = e[i] > 0.f ? side_of(fabs(real(i)), m, g) : side_of(fabsf(y[i]), m, g);
                w += (side > 0 || (side == 0 && (c & 1u)) ? 1u : 0u) << (4 * i);
            }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        w |= (y[i] < 0.f ? 8u : 0u) << (4 * i);
    return w;
}

// Element a (or with `second` b) of a pair at one position, in 64 bits.
// phase: the position's angle in turns of 2^-64.
__device__ __noinline__ double rotated_real(float a, float b, bool second, unsigned long long phase, float magnitude)
{
    double s, c;
    sincospi((double)(long long)phase * 0x1p-63, &s, &c);
    return (second ? (double)b * c + (double)a * s : (double)a * c - (double)b * s) * magnitude;
}

}  // namespace mercury
