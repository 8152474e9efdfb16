// quantize4.cuh -- blocks of 16 elements as e2m1 codes under an e4m3 scale.
//
// With g the head's scale, a block's scale is s = the e4m3 nearest to its
// largest magnitude over 6 |g|, and an element's code the e2m1 nearest to x /
// (s g), ties to even both times, of the real values: an element that was
// rotated is taken as its rotation is, not as 32 bits round it, so that what a
// cache holds does not hang on how sines are computed or sums are ordered.
//
// A value known to e (0 where it was not rotated) has its quotient bracketed by
// two 32-bit products, wider by 2^-21 than e, which covers their roundings (the
// reciprocal's 2^-23, and three of 2^-24); where both ends round to the same code, that is it.  Where they do
// not, the borders between the two are near the value, and it is compared with
// them: exactly in 32 bits, by the product's rounding error, or for a rotated
// value in 64 bits (one in some 10^5; as 0.2 % of warps meet one, that costs
// little).  There is one border mostly, and more where a rotation leaves a block
// far smaller than the elements that it was turned from (one half of a head
// small, and a small angle): e grows with those.
#pragma once
#include <stdint.h>

#include "paged.cuh"

namespace mercury {

// Eight floats as the nearest e2m1 codes (saturated at 6), the first in the
// lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&x)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// 1 / x to 2^-23 of it.
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Element a (or with `second` b) of a pair at one position, in 64 bits.
// phase: the position's angle in turns of 2^-64.
__device__ __noinline__ double rotated_real(float a, float b, bool second, unsigned long long phase, float magnitude)
{
    double s, c;
    sincospi((double)(long long)phase * 0x1p-63, &s, &c);
    return (second ? (double)b * c + (double)a * s : (double)a * c - (double)b * s) * magnitude;
}

// Where N elements of a block come from, for the rare ones that are settled in
// 64 bits: N of x, from element `at` of the head on, pairs of the plan's.
struct Source {
    const float *first, *second;  // of each element's pair
    unsigned long long pos;
    const unsigned long long *turns;
    float magnitude;
    int at, rot, interleaved;
    __device__ __forceinline__ double real(int i) const
    {
        const int j = at + i;
        if (j >= rot)  // a block may be turned in part
            return first[i];
        const int pair = interleaved ? j / 2 : j < rot / 2 ? j : j - rot / 2;
        return rotated_real(first[i], second[i], interleaved ? j & 1 : j >= rot / 2, turns[pair] * pos, magnitude);
    }
};

// Which of the scales' bytes lo to hi a block's is.  `from` where the elements
// were rotated: amax is then that of both halves of the block, y[N] this
// thread's half, and the threads of `both` settle it together.
template <int N>
__device__ __noinline__ uint32_t settle_scale(uint32_t lo, uint32_t hi, float amax, float off, float g, const float *y,
                                              const Source *from, unsigned int both)
{
    double x = 0.0;
    if (from) {
#pragma unroll 1
        for (int i = 0; i < N; ++i)
            if (fabsf(y[i]) + 2.f * off >= amax)  // it may be the largest
                x = fmax(x, fabs(from->real(i)));
        if (both) {
            __syncwarp(both);
            x = fmax(x, __shfl_xor_sync(both, x, 1));
        }
    }
#pragma unroll 1
    for (; lo < hi; ++lo) {
        const float m = 3.f * (e4m3_value(lo) + e4m3_value(lo + 1));  // 6 times the border above lo
        const int side = from ? side_of(x, m, g) : side_of(amax, m, g);
        if (side < 0 || (side == 0 && !(lo & 1u)))
            break;
    }
    return lo;
}

// The magnitudes lo with the codes settled that are others in hi, which has the
// elements' signs: a code is one of those between the two, and of a rotated
// element the sign, too, is that of its real value.  Returns the codes with
// signs.
__device__ __noinline__ uint32_t settle_codes(uint32_t lo, uint32_t hi, float s, float g, const float *y, const Source *from)
{
    uint32_t w = hi, differ = lo ^ (hi & 0x77777777u);
#pragma unroll 1
    while (differ) {
        const int i = (__ffs(differ) - 1) / 4, at = 4 * i;
        differ &= ~(15u << at);
        const double x = from ? from->real(i) : 0.0;
        uint32_t c = lo >> at & 7u, sign = hi >> at & 8u;
        for (const uint32_t most = hi >> at & 7u; c < most; ++c) {
            // the border above code c: 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5
            const float m = s * (c < 4 ? 0.5f * c + 0.25f : c < 6 ? (float)c - 1.5f : 5.f);
            const int side = from ? side_of(fabs(x), m, g) : side_of(fabsf(y[i]), m, g);
            if (side < 0 || (side == 0 && !(c & 1u)))
                break;
        }
        if (from)
            sign = x < 0.0 ? 8u : 0u;
        w = (w & ~(15u << at)) | (c | sign) << at;
    }
    return w;
}

// Largest magnitude, NaN where there is one.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The two ends' bytes for a block whose largest magnitude is amax, known to
// off: the lower end's in the lower byte.  (A NaN gives NaN, an infinity 448.)
__device__ __forceinline__ uint32_t scale_ends(float amax, float off, float g)
{
    const float r = reciprocal(6.f * g);
    return pack_e4m3((amax - off < 0.f ? 0.f : amax - off) * r * (1.f - kWider), (amax + off) * r * (1.f + kWider));
}

// Eight codes of four bits: the lower ends' magnitudes in lo, and in hi the
// upper ends' with the elements' signs.  s g: both scales; off: what the
// elements are known to.  Where s is zero all codes are.
__device__ __forceinline__ void code_ends(const float (&y)[8], float off, float s, float g, uint32_t &lo, uint32_t &hi)
{
    const float r = s > 0.f ? reciprocal(s * g) : 0.f;
    const float below = r * (1.f - kWider), above = r * (1.f + kWider);
    const float more = off * above * (1.f + kWider);
    float l[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        l[i] = fmaf(fabsf(y[i]), below, -more);
        h[i] = copysignf(fmaf(fabsf(y[i]), above, more), y[i]);
    }
    lo = pack_e2m1(l);
    const uint32_t less = lo & 0x88888888u;  // a lower end below zero is zero
    lo &= ~(less - (less >> 3)) & 0x77777777u;
    hi = pack_e2m1(h);
}

// Codes with signs as they are stored: all signs turned for a negative head
// scale, and a zero without one (which sign a zero's would be hangs on how 32
// bits round).
__device__ __forceinline__ uint32_t stored_codes(uint32_t w, float scale)
{
    const uint32_t magnitudes = w & 0x77777777u, some = (magnitudes + 0x77777777u) & 0x88888888u;
    return magnitudes | ((scale < 0.f ? ~w : w) & some);
}

}  // namespace mercury
