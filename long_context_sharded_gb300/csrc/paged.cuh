// paged.cuh -- what the rotary, cache-append and paged-attention kernels
// share: the rotation's angles, 8- and 16-bit conversions, and the view of a
// paged cache that a kernel gets by value.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mercury_attn.h"

namespace mercury {

// Error bit of the paged kernels' device error words: a length, position or
// page out of range (kErrBounds of ptx.cuh, here set in every build).
constexpr unsigned int kPagedErrBounds = 2u;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Launch chaining.  The serving kernels run a few microseconds each, one after
// another on a stream, so each may be brought onto the GPU while the kernel
// before it still runs (launch_chained) and waits for that kernel's end, and
// with it for everything earlier on the stream, before it touches memory.
// Every thread calls chain_wait first thing: a block that returned without it
// would let the grid end, and its successor begin, before the predecessor did.
__device__ __forceinline__ void chain_wait()
{
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

template <typename Args>
cudaError_t launch_chained(void (*kernel)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                           const Args &args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

// A tensor's element strides over (batch, head, token); the head dimension is
// contiguous.
struct Strides {
    long long b, h, s;
};

// A paged cache as a kernel sees it.
struct PagedView {
    char *k, *v;             // [num_pages][Hkv][page_size][d], pages page_stride elements apart
    const float *k_scale, *v_scale;  // [Hkv], 8-bit caches only
    const int *table;        // [B][max_pages], rows table_stride apart
    long long page_stride, table_stride;
    int Hkv, page_size, num_pages, max_pages;
    int page_shift;          // log2 of page_size, or -1 where it is no power of two
};

__device__ __forceinline__ int page_of(const PagedView &c, int pos)
{
    return c.page_shift >= 0 ? pos >> c.page_shift : (int)((unsigned int)pos / (unsigned int)c.page_size);
}

inline PagedView make_view(const mercury_paged_cache &c)
{
    PagedView v;
    v.k = (char *)c.k;
    v.v = (char *)c.v;
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.table = c.block_table;
    v.page_stride = c.page_stride;
    v.table_stride = c.table_stride;
    v.Hkv = c.Hkv;
    v.page_size = c.page_size;
    v.num_pages = c.num_pages;
    v.max_pages = c.max_pages;
    v.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (c.page_size == 1 << i)
            v.page_shift = i;
    return v;
}

// cos and sin of position * frequency, times the plan's magnitude.
//
// The frequency is held as turns per position in 64-bit fixed point, so the
// product with the position wraps modulo one turn exactly: no position, however
// far, costs the angle more than position * 2^-53 turns (the frequency's own
// rounding).  The product's upper 32 bits, as a signed fraction of a turn in
// [-1/2, 1/2), go to sincospif as x = 2 * fraction; rounding x to 24 bits is
// at most 2^-25 of half a turn, 1e-7 rad, which is what a 32-bit cosine keeps.
__device__ __forceinline__ void rope_cos_sin(unsigned long long turns, long long pos, float magnitude, float &c,
                                             float &s)
{
    const unsigned long long phase = turns * (unsigned long long)pos;
    const float x = (float)(int)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
    sincospif(x, &s, &c);
    s *= magnitude;
    c *= magnitude;
}

__device__ __forceinline__ float bf16_lo(uint32_t w)
{
    return __uint_as_float(w << 16);
}

__device__ __forceinline__ float bf16_hi(uint32_t w)
{
    return __uint_as_float(w & 0xffff0000u);
}

// Two floats rounded to nearest bf16, lo in the lower half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two floats rounded to nearest fp16, lo in the lower half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two floats rounded to nearest e4m3 and saturated at +-448, lo in the lower
// byte (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 bytes (the lower half of w) as fp16: exact.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

}  // namespace mercury
