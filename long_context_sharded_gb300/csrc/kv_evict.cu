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
// Rows are read once and written once; what is left is the selection, a chain
// of steps that each wait for the one before.
//
// Measured on a GB300: one sequence of 32K, 8 KV heads of 128, to 4K, 16 bits: 17
// us (5 us of bytes), 4 bits 14 (2); 16 sequences of 500 to 16K to 2K, 16 bits 53 us
// (40 us of bytes), 8 bits 35 (20), 4 bits 32 (12).  Each kernel alone and cold: selection 14 and 15 us, rows 10 and 23;
// with one block a head the first selection took 30 us.  32K tokens of a 4-bit
// cache read back: 29 us, 89 % of the measured copy bandwidth (8 bits 32 us, 95 %; 16
// bits 41, 98 %).
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mercury {

// Error word of this file's kernels: kPagedErrBounds = a length or page
// outside the table or the cache; the first site (0xa01 seq_lens, 0xa02 page,
// 0xa03 page of the shorter cache, 0xa04 head scales that differ).
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
constexpr int kMaxCluster = 8;
constexpr int kHeld = 32768;  // a block holds so many tokens' ranks in shared memory; of more it reads them anew

struct SelectArgs {
    const float *mass;  // [B][Hkv][width]
    const int *seq_lens;
    int *out_lens, *kept;  // [B], [B][Hkv][keep]
    float *out_mass;       // [B][Hkv][out_width], or none
    const unsigned int *scales[4];  // both caches' head scales of keys, then of values (bits), or none
    int Hkv, keep, first, last;
    int most;              // tokens that the table and mass can hold
    int held;              // ranks that a block holds
    long long width, out_width;
};

// A number's place in the order of all, -0 equal to 0.
__device__ __forceinline__ uint32_t rank_of_number(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// A weight's: NaN below everything.
__device__ __forceinline__ uint32_t rank_of(float x)
{
    return x != x ? 0u : rank_of_number(x);
}

// Inclusive scan over the block's 1024 threads.  `warps` is not used again
// before a barrier.
__device__ __forceinline__ int block_scan(int x, int *warps, int tid)
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
    const int sums = warps[lane];
    return x + __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The word, or four, at p of the cluster's block `rank`.
__device__ __forceinline__ int cluster_load(const int *p, uint32_t rank)
{
    int x;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.b32 %0, [a];\n\t}"
                 : "=r"(x)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return x;
}

__device__ __forceinline__ int4 cluster_load4(const int *p, uint32_t rank)
{
    int4 x;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return x;
}

// Rows are moved as they are, which gives them the same values under the same
// head scales only.  (Out of line, and in the kernel that selects: the one that
// moves has no registers to spare, one sequence of 32K took 17.8 us instead of 17.2.)
__device__ __noinline__ void look_at_scales(const SelectArgs &a, int h)
{
    if ((a.scales[0][h] ^ a.scales[1][h]) | (a.scales[2][h] ^ a.scales[3][h]))
        record_bounds(0xa04);
}

template <bool T>
struct Ties {
    static constexpr bool value = T;
};

constexpr int kListed = 4096;  // tokens of the first digit that are listed

struct __align__(16) SelectSmem {
    int bins[3][kBins];    // of each digit
    int halves[2][kBins];  // the cluster's, summed over half of its blocks each
    uint32_t list[kListed];
    int warps[6][kSelectWarps], found[3][3], counts[2], listed;
    uint4 ranks[1];        // [held / 4]
};

// A cluster of CS blocks a head of a sequence, each with a run of its tokens.
// The k-th largest rank is found digit by digit (11, 11 and 10 bits): a
// histogram in each block of those of its tokens that share the digits so far,
// summed by all blocks of the cluster, which then know the next digit.  Mostly
// few tokens share the first digit; those are listed, and the other two digits
// found by each block from all lists, which spares a pass over the tokens and
// two exchanges of histograms (5000 cycles each).  Then each block counts what
// it keeps, and each warp of it, and writes it behind what those before it keep.
// mass is read once, as ranks into shared memory.
// What bounds a head of 16K in one block is the integer unit: ends, NaN and
// ties looked at token by token it was busy 94 % (18 us; now 65 %, 15 us).
template <int CS>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ SelectArgs a)
{
    extern __shared__ __align__(16) char smem[];
    SelectSmem &sm = *reinterpret_cast<SelectSmem *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t me = CS > 1 ? cluster_rank() : 0u;
    for (int i = tid; i < 3 * kBins; i += kSelectThreads)
        (&sm.bins[0][0])[i] = 0;
    if (tid == 0)
        sm.listed = 0;
    chain_wait();
    const int bh = blockIdx.x / CS, b = bh / a.Hkv;
    const int given = a.seq_lens[b], n = min(max(given, 0), a.most);
    if (bh % a.Hkv == 0 && me == 0 && tid == 0) {
        if (given != n)
            record_bounds(0xa01);
        a.out_lens[b] = min(n, a.keep);
    }
    const float *const mass = a.mass + bh * a.width;
    int *const kept = a.kept + (long long)bh * a.keep;
    float *const out_mass = a.out_mass ? a.out_mass + bh * a.out_width : nullptr;
    if (a.scales[0] && n > 0 && me == 0 && tid == kSelectThreads - 1)
        look_at_scales(a, bh - b * a.Hkv);
    // this block's run: whole warps' runs of 128 tokens
    constexpr int LINE = 128;
    const int each = (n + CS * kSelectWarps * LINE - 1) / (CS * kSelectWarps * LINE) * LINE;  // of a warp
    const int from = min((int)me * each * kSelectWarps, n), to = min(from + each * kSelectWarps, n);
    if (n <= a.keep) {
        for (int i = from + tid; i < to; i += kSelectThreads) {
            kept[i] = i;
            if (out_mass)
                out_mass[i] = mass[i];
        }
        return;  // (all blocks of the cluster do)
    }
    // (keep >= first + last, and n > keep: the two ends do not meet.)  The ends
    // rank above every number.
    const int lo = a.first, hi = n - a.last;
    const bool held = to - from <= a.held;
    const bool quads = ((uintptr_t)mass & 15u) == 0;  // (runs begin at multiples of 128)
    // Of tokens i .. i + 3, whose weights are x where they all are numbers inside
    // the run and between the ends: 0 behind the run.
    auto inner = [&](int i) { return i >= lo && i + 4 <= hi && i + 4 <= to; };
    auto weights = [&](int i) {
        return quads ? *reinterpret_cast<const float4 *>(mass + i)
                     : make_float4(mass[i], mass[i + 1], mass[i + 2], mass[i + 3]);
    };
    auto ranks_of = [&](int i, float4 x, bool is_inner) {
        const float all = (x.x + x.y) + (x.z + x.w);  // NaN with one of them (and with infinities of both signs)
        if (is_inner && all == all)
            return make_uint4(rank_of_number(x.x), rank_of_number(x.y), rank_of_number(x.z), rank_of_number(x.w));
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            r[k] = i + k >= to ? 0u : i + k < lo || i + k >= hi ? 0xffffffffu : rank_of(mass[i + k]);
        return make_uint4(r[0], r[1], r[2], r[3]);
    };
    auto fetch = [&](int i) {
        const bool in = inner(i);
        return ranks_of(i, in ? weights(i) : make_float4(0.f, 0.f, 0.f, 0.f), in);
    };
    __syncthreads();  // the bins are zero
    auto ranks = [&](int i) { return held ? sm.ranks[(i - from) / 4] : fetch(i); };
    int want = a.keep;
    uint32_t prefix = 0;
    bool listed = false;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
        const int shift = kShift[pass], bits = kBits[pass];
        auto count = [&](uint32_t r) { atomicAdd(&sm.bins[pass][r >> shift & ((1u << bits) - 1u)], 1); };
        if (pass > 0 && listed) {
            // of the block warp / (kSelectWarps / CS)
            const uint32_t k = warp / (kSelectWarps / CS);
            const int many = CS > 1 ? cluster_load(&sm.listed, k) : sm.listed;
            for (int i = tid % (kSelectThreads / CS); i < many; i += kSelectThreads / CS) {
                const uint32_t r = CS > 1 ? (uint32_t)cluster_load((const int *)&sm.list[i], k) : sm.list[i];
                if (r >> (shift + bits) == prefix)
                    count(r);
            }
        } else if (pass == 0) {
            constexpr int U = 4;  // loads on their way
            for (int i0 = from + 4 * tid; i0 < to; i0 += U * 4 * kSelectThreads) {
                float4 w[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * 4 * kSelectThreads;
                    w[u] = inner(i) ? weights(i) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * 4 * kSelectThreads;
                    if (i >= to)
                        break;
                    const uint4 r = ranks_of(i, w[u], inner(i));
                    if (held)
                        sm.ranks[(i - from) / 4] = r;
                    const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (i + k < to)
                            count(x[k]);
                }
            }
        } else {
#pragma unroll 2
            for (int i = from + 4 * tid; i < to; i += 4 * kSelectThreads) {
                const uint4 r = ranks(i);
                const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (x[k] >> (shift + bits) == prefix && i + k < to)
                        count(x[k]);
            }
        }
        // from the top: thread t has the bins 2t' and 2t' + 1, t' = 1023 - t
        const int top = kBins - 1 - 2 * tid;
        int2 c;
        if (CS > 1 && !listed) {
            cluster_sync();
            // four bins of half of the blocks a thread
            int4 x[CS > 1 ? CS / 2 : 1];
            const int quad = tid % (kBins / 4) * 4, half = tid / (kBins / 4);
#pragma unroll
            for (int k = 0; k < CS / 2; ++k)
                x[k] = cluster_load4(&sm.bins[pass][quad], (me + half * (CS / 2) + k) % CS);
#pragma unroll
            for (int k = 1; k < CS / 2; ++k)
                x[0] = make_int4(x[0].x + x[k].x, x[0].y + x[k].y, x[0].z + x[k].z, x[0].w + x[k].w);
            *reinterpret_cast<int4 *>(&sm.halves[half][quad]) = x[0];
            __syncthreads();
            const int2 y = *reinterpret_cast<const int2 *>(&sm.halves[0][top - 1]);
            c = *reinterpret_cast<const int2 *>(&sm.halves[1][top - 1]);
            c = make_int2(c.x + y.x, c.y + y.y);
        } else {
            __syncthreads();
            c = *reinterpret_cast<const int2 *>(&sm.bins[pass][top - 1]);
        }
        const int incl = block_scan(c.x + c.y, sm.warps[pass], tid), before = incl - c.x - c.y;
        if (before < want && want <= incl) {
            const bool upper = before + c.y >= want;
            sm.found[pass][0] = upper ? top : top - 1;
            sm.found[pass][1] = upper ? before : before + c.y;
            sm.found[pass][2] = upper ? c.y : c.x;
        }
        __syncthreads();
        prefix = prefix << bits | (uint32_t)sm.found[pass][0];
        want -= sm.found[pass][1];
        if (pass == 0) {
            listed = sm.found[0][2] <= kListed;  // of all blocks
            if (listed) {
#pragma unroll 2
                for (int i = from + 4 * tid; i < to; i += 4 * kSelectThreads) {
                    const uint4 r = ranks(i);
                    const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (x[k] >> shift == prefix && i + k < to)
                            sm.list[atomicAdd(&sm.listed, 1)] = x[k];
                }
                if (CS > 1)
                    cluster_sync();
                else
                    __syncthreads();
            }
        }
    }
    const int first = from + warp * each, end = min(first + each, to);
    // Writes what is kept.  TIES: not all tokens at the threshold are, but the
    // first `ties` of them.
    auto write = [&](auto with_ties) {
        constexpr bool TIES = decltype(with_ties)::value;
        const int ties = want;
        // of a thread's four tokens: those above the threshold (without ties: or at
        // it, which is not 0 then), and those at it (in the upper half)
        auto look = [&](int i, uint32_t (&x)[4]) {
            const uint4 r = i < end ? ranks(i) : make_uint4(0, 0, 0, 0);
            x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
            int c = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!TIES)
                    c += x[k] >= prefix;
                else if (i + k < end)
                    c += (x[k] > prefix) + ((x[k] == prefix) << 16);
            return c;
        };
        int n_sure = 0, n_tie = 0;
#pragma unroll 2
        for (int i = first + 4 * lane; i - 4 * lane < end; i += LINE) {
            uint32_t x[4];
            const int c = look(i, x);
            n_sure += TIES ? c & 0xffff : c;
            n_tie += TIES ? c >> 16 : 0;
        }
        n_sure = __reduce_add_sync(0xffffffffu, n_sure);
        const int sure_incl = block_scan(lane == 0 ? n_sure : 0, sm.warps[3], tid);
        int at_sure = __shfl_sync(0xffffffffu, sure_incl - n_sure, 0), at_tie = 0;
        if (tid == kSelectThreads - 1)
            sm.counts[0] = sure_incl;
        if (TIES) {
            n_tie = __reduce_add_sync(0xffffffffu, n_tie);
            const int tie_incl = block_scan(lane == 0 ? n_tie : 0, sm.warps[4], tid);
            at_tie = __shfl_sync(0xffffffffu, tie_incl - n_tie, 0);
            if (tid == kSelectThreads - 1)
                sm.counts[1] = tie_incl;
        }
        if constexpr (CS > 1) {
            cluster_sync();
            const bool ahead = lane < (int)me;
            at_sure += __reduce_add_sync(0xffffffffu, ahead ? cluster_load(&sm.counts[0], lane) : 0);
            if (TIES)
                at_tie += __reduce_add_sync(0xffffffffu, ahead ? cluster_load(&sm.counts[1], lane) : 0);
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        }
        for (int i = first + 4 * lane; i - 4 * lane < end; i += LINE) {
            uint32_t x[4];
            const int c = look(i, x);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += y;
            }
            const int all = __shfl_sync(0xffffffffu, incl, 31);
            int sure = at_sure + (TIES ? (incl & 0xffff) - (c & 0xffff) : incl - c), tie = TIES ? at_tie + (incl >> 16) - (c >> 16) : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bool stays;
                int slot;
                if (TIES) {
                    const bool above = x[k] > prefix, at = x[k] == prefix, in = i + k < end;
                    stays = in && (above || (at && tie < ties));
                    slot = sure + min(tie, ties);
                    sure += in && above;
                    tie += in && at;
                } else {
                    stays = x[k] >= prefix;
                    slot = sure;
                    sure += stays;
                }
                if (stays) {
                    kept[slot] = i + k;
                    if (out_mass)  // (an end's rank, NaN's and a zero's is not its weight's own)
                        out_mass[slot] = x[k] == 0xffffffffu || x[k] == 0u || x[k] == 0x80000000u
                                             ? mass[i + k]
                                             : __uint_as_float(x[k] & 0x80000000u ? x[k] ^ 0x80000000u : ~x[k]);
                }
            }
            at_sure += TIES ? all & 0xffff : all;
            at_tie += TIES ? all >> 16 : 0;
        }
    };
    // (without ties the threshold is above 0: else all tokens would stay)
    if (sm.found[2][2] == want)
        write(Ties<false>());
    else
        write(Ties<true>());
    if constexpr (CS > 1)  // a block's counts and list are read until here
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int CS>
int prepare_select(char *msg, size_t msg_len)
{
    KernelInfo ki;
    return prepare_kernel((const void *)evict_select_kernel<CS>, (int)sizeof(SelectSmem) + kHeld * 4, &ki, msg, msg_len);
}

template <int CS>
int launch_select(SelectArgs &s, long long heads, cudaStream_t stream, char *msg, size_t msg_len)
{
    const int line = CS * kSelectWarps * 128, run = ((s.most - 1) / line + 1) * (kSelectWarps * 128);
    s.held = run < kHeld ? run : kHeld;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(heads * CS));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = sizeof(SelectSmem) + s.held * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {CS, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = CS > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel<CS>, s);
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "cache eviction launch: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

// ------------------------------------------------------------------ and their rows

constexpr int kMoveThreads = 256;
// Rows that a thread has on the way, of keys and of values: more of them leave
// fewer blocks (16 sequences to 2K, the slower selection before: 36 us with 2, 38
// with 1, 39 with 4, 48 with 8).
constexpr int kMoveAhead = 2;

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
            from[i] = page * s.page_stride +
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
        for (int i = 0; i < 2; ++i) {
            o[4 * i] = scaled_bf16(mul_f16(e2m1_to_f16<0>(w[i]), s2), scale);
            o[4 * i + 1] = scaled_bf16(mul_f16(e2m1_to_f16<1>(w[i]), s2), scale);
            o[4 * i + 2] = scaled_bf16(mul_f16(e2m1_to_f16<2>(w[i]), s2), scale);
            o[4 * i + 3] = scaled_bf16(mul_f16(e2m1_to_f16<3>(w[i]), s2), scale);
        }
    }
};

// 16 elements: a whole sector where the output allows it (two stores of 16
// bytes each write half of one).
__device__ __forceinline__ void store_block(__nv_bfloat16 *p, const uint32_t (&o)[8])
{
    if (((uintptr_t)p & 31u) == 0) {
        st_global_v8(p, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(p + 8) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

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
        store_block(a.k + to, o);
        y[i].widen(o, vs);
        store_block(a.v + to, o);
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
    SelectArgs s = {};
    s.mass = mass;
    s.seq_lens = seq_lens;
    s.out_lens = out_lens;
    s.kept = kept;
    s.out_mass = out_mass;
    s.Hkv = cache.Hkv;
    s.keep = keep;
    s.first = first;
    s.last = last;
    s.most = (int)(held < width ? held : width);
    s.width = width;
    s.out_width = out_width;
    if (cache.elem != MERCURY_ELEM_BF16) {
        s.scales[0] = (const unsigned int *)cache.k_scale;
        s.scales[1] = (const unsigned int *)into.k_scale;
        s.scales[2] = (const unsigned int *)cache.v_scale;
        s.scales[3] = (const unsigned int *)into.v_scale;
    }
    const long long heads = (long long)cache.B * cache.Hkv;
    if (heads * kMaxCluster > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many heads for one call (%lld)", heads);
        return MERCURY_EINVAL;
    }
    // As many blocks of a head as leave one for each SM, where each gets 2K
    // tokens or more.
    int sms = 0;
    int rc = device_sm_count(&sms);
    // (all of them, so that a call of other sizes may be captured)
    if (rc == MERCURY_OK)
        rc = prepare_select<1>(msg, msg_len);
    if (rc == MERCURY_OK)
        rc = prepare_select<2>(msg, msg_len);
    if (rc == MERCURY_OK)
        rc = prepare_select<4>(msg, msg_len);
    if (rc == MERCURY_OK)
        rc = prepare_select<8>(msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    rc = heads * 8 <= sms && s.most > 8192   ? launch_select<8>(s, heads, stream, msg, msg_len)
         : heads * 4 <= sms && s.most > 4096 ? launch_select<4>(s, heads, stream, msg, msg_len)
         : heads * 2 <= sms && s.most > 2048 ? launch_select<2>(s, heads, stream, msg, msg_len)
                                             : launch_select<1>(s, heads, stream, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
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
