// kv_evict.cu -- a sequence's heaviest keys and values into a shorter cache, and
// a cache read back as 16-bit keys and values.
//
// Eviction.  Of sequence b's n = seq_lens[b] cached tokens each KV head keeps
// min(n, keep): the first `first`, the last `last`, and of the others those
// with the most of mass[b][h][:], of two equal ones the earlier.  They keep
// their order: token j of the shorter cache is token kept[b][h][j].
//
// Reading back.  k_out[b][h][i] = the values of token i's row, rounded once.
//
// Both are bound by memory: a row is read once and written once.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mercury {

// Error word of this file's kernels: kPagedErrBounds = a length or page
// outside the table or the cache; the first site (0xa01 seq_lens, 0xa02 page,
// 0xa03 page of the shorter cache).
__device__ unsigned int g_evict_err_word = 0;
__device__ unsigned int g_evict_err_site = 0;

namespace {

__device__ __noinline__ void record_bounds(unsigned int site)
{
    atomicOr(&g_evict_err_word, kPagedErrBounds);
    atomicCAS(&g_evict_err_site, 0u, site);
}

// ------------------------------------------------------------------ which tokens are kept

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;

struct SelectArgs {
    const float *mass;  // [B][Hkv][width]
    const int *seq_lens;
    int *out_lens, *kept;  // [B], [B][Hkv][keep]
    float *out_mass;       // [B][Hkv][out_width], or none
    int Hkv, keep, first, last;
    int most;              // tokens that the table and mass can hold
    long long width, out_width;
};

// A weight's place in the order of all: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t rank_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive scan over the block's 1024 threads; total: of all of them.
__device__ __forceinline__ int block_scan(int x, int *warps, int tid, int &total)
{
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        warps[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o)
                w += y;
        }
        warps[lane] = w;
    }
    __syncthreads();
    total = warps[kSelectWarps - 1];
    x += warp ? warps[warp - 1] : 0;
    __syncthreads();
    return x;
}

// A block a head of a sequence.  The k-th largest rank is found digit by digit
// (11, 11 and 10 bits), from a histogram of the tokens that share the digits so
// far; then each warp counts, and after a scan writes, its run of the tokens.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ SelectArgs a)
{
    __shared__ int bins[kBins];
    __shared__ int warps[kSelectWarps], found[2];
    chain_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x, b = bh / a.Hkv;
    const int given = a.seq_lens[b], n = min(max(given, 0), a.most);
    const int m = min(n, a.keep);
    if (bh % a.Hkv == 0 && tid == 0) {
        if (given != n)
            record_bounds(0xa01);
        a.out_lens[b] = m;
    }
    const float *const mass = a.mass + bh * a.width;
    int *const kept = a.kept + (long long)bh * a.keep;
    float *const out_mass = a.out_mass ? a.out_mass + bh * a.out_width : nullptr;
    if (n <= a.keep) {
        for (int i = tid; i < n; i += kSelectThreads) {
            kept[i] = i;
            if (out_mass)
                out_mass[i] = mass[i];
        }
        return;
    }
    // (keep >= first + last, and n > keep: the two ends do not meet)
    const int lo = a.first, hi = n - a.last;
    int want = a.keep - a.first - a.last;  // of the others
    uint32_t prefix = 0;
    int ties = 0;                          // tokens at the threshold that are kept
    if (want > 0) {
        int shift = 21, bits = 11;
        for (int pass = 0; pass < 3; ++pass) {
            for (int i = tid; i < kBins; i += kSelectThreads)
                bins[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kSelectThreads) {
                const uint32_t r = rank_of(mass[i]);
                if (pass == 0 || r >> (shift + bits) == prefix)
                    atomicAdd(&bins[r >> shift & ((1u << bits) - 1u)], 1);
            }
            __syncthreads();
            // from the top: thread t has the bins 2t' and 2t' + 1, t' = 1023 - t
            const int top = kBins - 1 - 2 * tid;
            const int c1 = bins[top], c0 = bins[top - 1];
            int total;
            const int incl = block_scan(c0 + c1, warps, tid, total), before = incl - c0 - c1;
            if (before < want && want <= incl) {
                const bool upper = before + c1 >= want;
                found[0] = upper ? top : top - 1;
                found[1] = upper ? before : before + c1;
            }
            __syncthreads();
            prefix = prefix << bits | (uint32_t)found[0];
            want -= found[1];
            const int next = pass == 1 ? 10 : 11;
            __syncthreads();
            if (pass < 2) {
                bits = pass == 0 ? 11 : next;
                shift -= bits;
            }
        }
        ties = want;
    } else {
        prefix = 0xffffffffu;  // (no weight ranks above it)
    }
    const bool none = a.keep == a.first + a.last;
    // each warp's run of tokens
    const int each = (n + kSelectWarps * 32 - 1) / (kSelectWarps * 32) * 32, from = min(warp * each, n),
              to = min(from + each, n);
    auto look = [&](int i, bool &sure, bool &tie) {
        sure = tie = false;
        if (i < to) {
            const bool end = i < lo || i >= hi;
            const uint32_t r = end || none ? 0u : rank_of(mass[i]);
            sure = end || (!none && r > prefix);
            tie = !end && !none && r == prefix;
        }
    };
    int n_sure = 0, n_tie = 0;
    for (int i = from; i < to; i += 32) {
        bool sure, tie;
        look(i + lane, sure, tie);
        n_sure += __popc(__ballot_sync(0xffffffffu, sure));
        n_tie += __popc(__ballot_sync(0xffffffffu, tie));
    }
    int total;
    int at_sure = block_scan(lane == 0 ? n_sure : 0, warps, tid, total) - n_sure;
    int at_tie = block_scan(lane == 0 ? n_tie : 0, warps, tid, total) - n_tie;
    at_sure = __shfl_sync(0xffffffffu, at_sure, 0);
    at_tie = __shfl_sync(0xffffffffu, at_tie, 0);
    const unsigned below = (1u << lane) - 1u;
    for (int i = from; i < to; i += 32) {
        bool sure, tie;
        look(i + lane, sure, tie);
        const unsigned s = __ballot_sync(0xffffffffu, sure), t = __ballot_sync(0xffffffffu, tie);
        const int rank = at_tie + __popc(t & below);  // of the ties before this one
        if (sure || (tie && rank < ties)) {
            const int slot = at_sure + __popc(s & below) + min(rank, ties);
            kept[slot] = i + lane;
            if (out_mass)
                out_mass[slot] = mass[i + lane];
        }
        at_sure += __popc(s);
        at_tie += __popc(t);
    }
}

// ------------------------------------------------------------------ and their rows

constexpr int kMoveThreads = 256;
constexpr int kMoveAhead = 4;  // rows that a thread has on the way, of keys and of values

struct MoveArgs {
    PagedView src, dst;
    const int *lens, *kept;  // of the shorter cache
    int keep, chunks;        // rows of a head, blocks for them
    int Hkv;
};

// Rows of UNITS units of type U.  A block has a run of the kept tokens of a head
// of a sequence.
template <typename U, int UNITS>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ MoveArgs a)
{
    constexpr int ROWS = kMoveThreads / UNITS;  // at a time
    chain_wait();
    const int chunk = blockIdx.x % a.chunks, bh = blockIdx.x / a.chunks, b = bh / a.Hkv, h = bh % a.Hkv;
    const int unit = threadIdx.x % UNITS, row = threadIdx.x / UNITS;
    const int n = a.lens[b], base = chunk * (ROWS * kMoveAhead);
    if (row >= ROWS || base >= n)
        return;
    const PagedView &s = a.src, &d = a.dst;
    long long from[kMoveAhead], to[kMoveAhead];  // bytes; -1: not there
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i) {
        const int slot = base + i * ROWS + row;
        from[i] = to[i] = -1;
        if (slot >= n)
            continue;
        const int token = a.kept[(long long)bh * a.keep + slot];
        const int sp = page_of(s, token);
        const int page = s.table[b * s.table_stride + sp];
        if (page >= 0 && page < s.num_pages)
            from[i] = page * s.page_stride * (long long)1 +
                      ((long long)h * s.page_size + token - sp * s.page_size) * (UNITS * sizeof(U));
        else
            record_bounds(0xa02);
        const int dp = page_of(d, slot);
        const int into = dp < d.max_pages ? d.table[b * d.table_stride + dp] : -1;
        if (into >= 0 && into < d.num_pages)
            to[i] = into * d.page_stride + ((long long)h * d.page_size + slot - dp * d.page_size) * (UNITS * sizeof(U));
        else
            record_bounds(0xa03);
    }
    U x[kMoveAhead], y[kMoveAhead];
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i) {
        x[i] = y[i] = U();
        if (from[i] >= 0 && to[i] >= 0) {
            x[i] = reinterpret_cast<const U *>(s.k + from[i])[unit];
            y[i] = reinterpret_cast<const U *>(s.v + from[i])[unit];
        }
    }
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i)
        if (to[i] >= 0) {  // a token whose page does not exist counts as zeros
            reinterpret_cast<U *>(d.k + to[i])[unit] = x[i];
            reinterpret_cast<U *>(d.v + to[i])[unit] = y[i];
        }
}

template <typename U, int UNITS>
int launch_move(MoveArgs &a, int B, cudaStream_t stream, char *msg, size_t msg_len)
{
    constexpr int each = kMoveThreads / UNITS * kMoveAhead;
    a.chunks = (a.keep + each - 1) / each;
    const long long blocks = (long long)a.chunks * B * a.Hkv;
    if (blocks > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many tokens for one call (%lld)", blocks * each);
        return MERCURY_EINVAL;
    }
    const cudaError_t e =
        launch_chained(evict_move_kernel<U, UNITS>, dim3((unsigned)blocks), kMoveThreads, 0, stream, a);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache eviction launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

// ------------------------------------------------------------------ reading back

constexpr int kReadThreads = 256;
constexpr int kReadAhead = 4;

struct ReadArgs {
    PagedView cache;
    const int *seq_lens;
    __nv_bfloat16 *k, *v;  // [B][Hkv][S][d]
    int S, chunks;
};

// 16 elements of a row, as they are held.
template <int ELEM>
struct Held;

template <>
struct Held<MERCURY_ELEM_BF16> {
    uint4 w[2];
    __device__ __forceinline__ void load(const char *row, int blk, int)
    {
        w[0] = reinterpret_cast<const uint4 *>(row)[2 * blk];
        w[1] = reinterpret_cast<const uint4 *>(row)[2 * blk + 1];
    }
    __device__ __forceinline__ void widen(uint32_t (&o)[8], float) const
    {
        o[0] = w[0].x, o[1] = w[0].y, o[2] = w[0].z, o[3] = w[0].w;
        o[4] = w[1].x, o[5] = w[1].y, o[6] = w[1].z, o[7] = w[1].w;
    }
};

__device__ __forceinline__ uint32_t scaled_bf16(uint32_t f16, float s)
{
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&f16));
    return pack_bf16(x.x * s, x.y * s);
}

template <>
struct Held<MERCURY_ELEM_E4M3> {
    uint4 w;
    __device__ __forceinline__ void load(const char *row, int blk, int) { w = reinterpret_cast<const uint4 *>(row)[blk]; }
    __device__ __forceinline__ void widen(uint32_t (&o)[8], float scale) const
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = scaled_bf16(e4m3_to_f16(x[i]), scale);
            o[2 * i + 1] = scaled_bf16(e4m3_to_f16(x[i] >> 16), scale);
        }
    }
};

template <>
struct Held<MERCURY_ELEM_E2M1> {
    uint32_t w[2], s;
    __device__ __forceinline__ void load(const char *row, int blk, int d)
    {
        // (rows of 36 bytes: words)
        w[0] = reinterpret_cast<const uint32_t *>(row)[2 * blk];
        w[1] = reinterpret_cast<const uint32_t *>(row)[2 * blk + 1];
        s = *reinterpret_cast<const uint8_t *>(row + d / 2 + blk);
    }
    __device__ __forceinline__ void widen(uint32_t (&o)[8], float scale) const
    {
        // code times scale is exact in fp16; times the head's, rounded to 32
        // bits and then once more
        const uint32_t s2 = e4m3_to_f16(s | s << 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t byte = w[i / 4] >> (8 * (i % 4)) & 0xffu;
            uint32_t x;
            asm("{\n\t.reg .b8 lo, hi;\n\tmov.b16 {lo, hi}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, lo;\n\tmul.rn.f16x2 %0, %0, %2;\n\t}"
                : "=r"(x)
                : "h"((uint16_t)byte), "r"(s2));
            o[i] = scaled_bf16(x, scale);
        }
    }
};

template <int ELEM, int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const __grid_constant__ ReadArgs a)
{
    constexpr int BLKS = D / 16, TOKENS = kReadThreads / BLKS;  // at a time
    constexpr int ROWB = ELEM == MERCURY_ELEM_BF16 ? 2 * D : ELEM == MERCURY_ELEM_E4M3 ? D : D / 2 + D / 16;
    chain_wait();
    const PagedView &c = a.cache;
    const int chunk = blockIdx.x % a.chunks, bh = blockIdx.x / a.chunks, b = bh / c.Hkv, h = bh % c.Hkv;
    const int given = a.seq_lens[b], n = min(min(max(given, 0), c.max_pages * c.page_size), a.S);
    if (given != n && chunk == 0 && h == 0 && threadIdx.x == 0)
        record_bounds(0xa01);
    const int blk = threadIdx.x % BLKS, base = chunk * (TOKENS * kReadAhead) + threadIdx.x / BLKS;
    if (base >= n)
        return;
    const float ks = ELEM == MERCURY_ELEM_BF16 ? 1.f : c.k_scale[h], vs = ELEM == MERCURY_ELEM_BF16 ? 1.f : c.v_scale[h];
    Held<ELEM> x[kReadAhead], y[kReadAhead];
    bool there[kReadAhead];
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
        const int token = base + i * TOKENS;
        x[i] = y[i] = Held<ELEM>{};
        there[i] = token < n;
        if (!there[i])
            continue;
        const int p = page_of(c, token), page = c.table[b * c.table_stride + p];
        if (page >= 0 && page < c.num_pages) {
            const long long at = page * c.page_stride * (ELEM == MERCURY_ELEM_BF16 ? 2 : 1) +
                                 ((long long)h * c.page_size + token - p * c.page_size) * ROWB;
            x[i].load(c.k + at, blk, D);
            y[i].load(c.v + at, blk, D);
        } else {
            record_bounds(0xa02);  // such a token counts as zeros
        }
    }
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
        if (!there[i])
            continue;
        const long long to = ((long long)bh * a.S + base + i * TOKENS) * D + blk * 16;
        uint32_t o[8];
        x[i].widen(o, ks);
        *reinterpret_cast<uint4 *>(a.k + to) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(a.k + to + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        y[i].widen(o, vs);
        *reinterpret_cast<uint4 *>(a.v + to) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(a.v + to + 8) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

template <int ELEM, int D>
int launch_read(ReadArgs &a, int B, cudaStream_t stream, char *msg, size_t msg_len)
{
    constexpr int each = kReadThreads / (D / 16) * kReadAhead;
    a.chunks = (a.S + each - 1) / each;
    const long long blocks = (long long)a.chunks * B * a.cache.Hkv;
    if (blocks > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many tokens for one call (%lld)", blocks * each);
        return MERCURY_EINVAL;
    }
    const cudaError_t e = launch_chained(kv_read_kernel<ELEM, D>, dim3((unsigned)blocks), kReadThreads, 0, stream, a);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache read launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

template <int D>
int launch_read_elem(ReadArgs &a, int elem, int B, cudaStream_t stream, char *msg, size_t msg_len)
{
    return elem == MERCURY_ELEM_BF16   ? launch_read<MERCURY_ELEM_BF16, D>(a, B, stream, msg, msg_len)
           : elem == MERCURY_ELEM_E4M3 ? launch_read<MERCURY_ELEM_E4M3, D>(a, B, stream, msg, msg_len)
                                       : launch_read<MERCURY_ELEM_E2M1, D>(a, B, stream, msg, msg_len);
}

}  // namespace

int launch_kv_evict(const mercury_paged_cache &cache, const mercury_paged_cache &into, const float *mass, long long width,
                    const int *seq_lens, int keep, int first, int last, int *out_lens, int *kept, float *out_mass,
                    long long out_width, cudaStream_t stream, char *msg, size_t msg_len)
{
    const long long held = (long long)cache.max_pages * cache.page_size;
    SelectArgs s = {mass, seq_lens, out_lens, kept, out_mass, cache.Hkv, keep, first, last,
                    (int)(held < width ? held : width), width, out_width};
    const long long heads = (long long)cache.B * cache.Hkv;
    if (heads > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many heads for one call (%lld)", heads);
        return MERCURY_EINVAL;
    }
    const cudaError_t e =
        launch_chained(evict_select_kernel, dim3((unsigned)heads), kSelectThreads, 0, stream, s);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache eviction launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    MoveArgs a;
    a.src = make_view(cache);
    a.dst = make_view(into);
    if (cache.elem == MERCURY_ELEM_BF16) {  // strides in bytes
        a.src.page_stride *= 2;
        a.dst.page_stride *= 2;
    }
    a.lens = out_lens;
    a.kept = kept;
    a.keep = keep;
    a.Hkv = cache.Hkv;
    const bool wide = cache.d == 128;
    if (cache.elem == MERCURY_ELEM_BF16)
        return wide ? launch_move<uint4, 16>(a, cache.B, stream, msg, msg_len)
                    : launch_move<uint4, 8>(a, cache.B, stream, msg, msg_len);
    if (cache.elem == MERCURY_ELEM_E4M3)
        return wide ? launch_move<uint4, 8>(a, cache.B, stream, msg, msg_len)
                    : launch_move<uint4, 4>(a, cache.B, stream, msg, msg_len);
    return wide ? launch_move<uint2, 9>(a, cache.B, stream, msg, msg_len)
                : launch_move<uint32_t, 9>(a, cache.B, stream, msg, msg_len);
}

int launch_kv_read(const mercury_paged_cache &cache, const int *seq_lens, int S, void *k, void *v, cudaStream_t stream,
                   char *msg, size_t msg_len)
{
    ReadArgs a;
    a.cache = make_view(cache);
    a.seq_lens = seq_lens;
    a.k = (__nv_bfloat16 *)k;
    a.v = (__nv_bfloat16 *)v;
    a.S = S;
    return cache.d == 128 ? launch_read_elem<128>(a, cache.elem, cache.B, stream, msg, msg_len)
                          : launch_read_elem<64>(a, cache.elem, cache.B, stream, msg, msg_len);
}

int read_and_clear_evict_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    return read_and_clear_words(g_evict_err_word, g_evict_err_site, "cache eviction", word, site, msg, msg_len);
}

}  // namespace mercury
