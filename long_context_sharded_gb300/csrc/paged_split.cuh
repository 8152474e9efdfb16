// paged_split.cuh -- what the kernels of attention over a paged cache share: the
// line of all jobs' tiles and its equal shares, a block's bounded waits, the
// matrix instruction and the terms that a weight enters it as, and the second
// kernel, which joins the parts of jobs that were cut between blocks.
//
// Everything here has internal linkage: each file that includes it has error
// words of its own.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mercury {
namespace {

// Error word of this file's kernels: kPagedErrBounds = a length or page
// outside the table or the cache, kErrTimeout = a bounded wait ran out; the
// first site (0x901 seq_lens, 0x902 new_lens, 0x903 page, 0x904 wait).
__device__ unsigned int g_paged_err_word = 0;
__device__ unsigned int g_paged_err_site = 0;

constexpr int kCopyWarps = 4;                // and those that copy
constexpr int kJoinWarps = 8;                // of a block of the second kernel
constexpr int kJoinAhead = 4;                // parts that each has on the way
constexpr uint32_t kEndBarrier = 15;         // named barrier at a block's end

struct PagedArgs {
    CUtensorMap map_k, map_v;  // the cache in boxes of box_rows keys, where box_rows > 0
    const __nv_bfloat16 *q;
    Strides qs;
    PagedView cache;
    const int *seq_lens, *new_lens;
    void *out;
    float *lse;
    float *ws_o;    // [2 * blocks][rows of a tile][d]: unnormalised sums of a part
    float2 *ws_ml;  // [2 * blocks][rows of a tile]: maximum (log2 units), sum of exponentials
    int4 *ws_rec;   // [blocks]: job cut behind its first part in the block, its new tokens, -, its last
                    // block (-1: none)
    int B, Hq, Hkv, G, Sq, R, n_rt, causal, out_bf16;
    int join_warps; // warps for a row there
    int box_rows;   // keys of a tensor copy: the largest power of two that divides page_size, at most a
                    // tile; 0 below 8 (the rows of a swizzle), where keys are copied one by one, which
                    // takes longer (pages of 8, one by one: 16 of 700 to 32K 174 us instead of 170, 8-bit
                    // 84 instead of 78, 64 short ones 55.7 instead of 50.5)
    float scale_log2;
    int fault;      // test hook: withhold one copying warp's copies
    unsigned long long wait_ns;
};

__device__ __forceinline__ void record_bounds(unsigned int site)
{
    atomicOr(&g_paged_err_word, kPagedErrBounds);
    atomicCAS(&g_paged_err_site, 0u, site);
}

// A block's end.  A wait that runs out sets `now`: no copy is sent after that
// and no further wait lasts; the computing warps walk on to the end with
// whatever data there is, since which tiles, rows and barriers they touch does
// not depend on it.  `sent`: tiles that each copying warp has sent.
struct Stop {
    int now;
    int sent[kCopyWarps];
};

__device__ __forceinline__ bool stopped(const Stop *stop)
{
    return *reinterpret_cast<const volatile int *>(&stop->now) != 0;
}

// Waits for a phase of `bar`, at most `limit` ns, or until the block stops.
__device__ __forceinline__ void wait_long(uint64_t *bar, uint32_t parity, unsigned long long limit, Stop *stop)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (stopped(stop))
            return;
        if (globaltimer_ns() - t0 > limit) {
            *reinterpret_cast<volatile int *>(&stop->now) = 1;
            atomicOr(&g_paged_err_word, kErrTimeout);
            atomicCAS(&g_paged_err_site, 0u, 0x904u);
            return;
        }
    }
}

__device__ __forceinline__ void wait_phase(uint64_t *bar, uint32_t parity, unsigned long long limit, Stop *stop)
{
    if (!mbar_try_wait(bar, parity))
        wait_long(bar, parity, limit, stop);
}

// Arrive on a named barrier without waiting.
__device__ __forceinline__ void named_barrier_arrive(uint32_t id, uint32_t nthreads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8); bf16 operands, or fp16 for an
// 8-bit cache.
template <bool F16>
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B.
template <bool F16>
__device__ __forceinline__ void mma_first(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// o += d f, rounded to nearest, two elements an instruction (28 rows of 128 at
// 20K to 32K keys: 3 % less time than one by one).
__device__ __forceinline__ void add_to(float *o, const float *d, float f)
{
#pragma unroll
    for (int e = 0; e < 4; e += 2)
        asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmov.b64 z, {%4, %4};\n\t"
            "fma.rn.f32x2 x, y, z, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
            : "+f"(o[e]), "+f"(o[e + 1])
            : "f"(d[e]), "f"(d[e + 1]), "f"(f));
}

// p as a sum of 16-bit terms, each the nearest to what those before it leave.
// Three bf16 ones hold it to 2^-26.  (Two, 2^-18, left O four times further from
// 64 bits than a 32-bit softmax does.)
//
// Of two fp16 ones the second is kept 2^kLowShift times as large, with sums of
// its own: fp16 ends at 2^-24, and a weight far below the largest, or the rest
// of one, would lose its bits there, as every key does beside a sink (16K keys
// 17 nats below one, 8 rows: their part of O 5 % off; now 2e-6).  For the same
// reason weights are taken 2^kUp times as large, with a maximum that is raised
// already by scores 2^kGrow above it, so that they fill fp16's upper half.
// They are held to 2^-23, and the smallest ones to 2^-48 of the largest.
constexpr int kLowShift = 11;
template <bool F16>
constexpr float kGrow = F16 ? 3.f : 8.f;
template <bool F16>
constexpr float kUp = F16 ? 12.f : 0.f;
constexpr float kLow = 1.f / (1 << kLowShift);
template <bool F16>
__device__ __forceinline__ void split(float p0, float p1, uint32_t (&term)[F16 ? 2 : 3])
{
    if constexpr (F16) {
        term[0] = pack_f16(p0, p1);
        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&term[0]));
        term[1] = pack_f16((p0 - h.x) * (1 << kLowShift), (p1 - h.y) * (1 << kLowShift));
    } else {
        term[0] = pack_bf16(p0, p1);
        p0 -= bf16_lo(term[0]);
        p1 -= bf16_hi(term[0]);
        term[1] = pack_bf16(p0, p1);
        term[2] = pack_bf16(p0 - bf16_lo(term[1]), p1 - bf16_hi(term[1]));
    }
}

__device__ __forceinline__ int keys_of(const PagedArgs &a, int b)
{
    const int most = a.cache.max_pages * a.cache.page_size;
    return min(max(a.seq_lens[b], 0), most);
}

__device__ __forceinline__ int new_of(const PagedArgs &a, int b)
{
    return a.new_lens ? min(max(a.new_lens[b], 0), a.Sq) : a.Sq;
}

// Positions.  All jobs lie on one line, in units of an eighth of a tile, the
// time that its keys take: a full tile is eight, a job's last one as many as
// it has eighths, and a job takes kJobCost more before its first tile, what
// changing jobs costs a block (64 sequences of 1 to 2047 tokens, 16 heads of
// 64: 53.5 us with 4 units, 50.8 with 7, 49.4 with 10 and 14; of 1 to 600
// tokens 36.7, 30.3, 27.9 and 26.1).  A tile
// belongs to the share that holds its first unit.
constexpr int kUnits = 8;
constexpr int kJobCost = 14;

// A tile on that line.
struct Place {
    int pos;          // its first unit
    int b, hr, j;     // sequence, job (KV head * row tiles + row tile), tile of the job
    int tiles, keys;  // of sequence b: tiles of a job, keys
};

template <int TILE>
__device__ __forceinline__ int tiles_of(int keys, int n)
{
    return n > 0 ? max(1, (keys + TILE - 1) / TILE) : 0;
}

template <int TILE>
__device__ __forceinline__ void enter(const PagedArgs &a, Place &p)
{
    p.keys = keys_of(a, p.b);
    p.tiles = tiles_of<TILE>(p.keys, new_of(a, p.b));
}

// Units of a job's last tile.
template <int TILE>
__device__ __forceinline__ int last_units(int keys, int tiles)
{
    return max(1, (keys - (tiles - 1) * TILE + TILE / kUnits - 1) / (TILE / kUnits));
}

// First unit of the tile behind p (of the next job's first one, if there is one).
template <int TILE>
__device__ __forceinline__ int next_pos(const Place &p)
{
    return p.pos + (p.j + 1 < p.tiles ? kUnits : last_units<TILE>(p.keys, p.tiles) + kJobCost);
}

// The tile at `pos`, the one behind p.
template <int TILE>
__device__ __forceinline__ void advance(const PagedArgs &a, Place &p, int pos)
{
    p.pos = pos;
    if (++p.j < p.tiles)
        return;
    p.j = 0;
    if (++p.hr < a.Hkv * a.n_rt)
        return;
    p.hr = 0;
    do {
        ++p.b;  // there is one: the position lies before the share's end
        enter<TILE>(a, p);
    } while (p.tiles == 0);
}

// (Loads of what an earlier kernel may have written are plain ones: the
// read-only path promises nothing about data that was written after this
// kernel came up.)

// The line in equal shares: block c has [first(c), first(c + 1)).
struct Shares {
    int each, more;  // positions of every share, and shares with one more
    __device__ __forceinline__ int first(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int owner(int pos) const
    {
        const int longer = more * (each + 1);
        return pos < longer ? pos / (each + 1) : more + (pos - longer) / each;
    }
};

// Positions of all jobs of sequence b (0 behind the last).
template <int TILE>
__device__ __forceinline__ int length_of(const PagedArgs &a, int b)
{
    if (b >= a.B)
        return 0;
    const int keys = keys_of(a, b), tiles = tiles_of<TILE>(keys, new_of(a, b));
    return tiles == 0 ? 0 : (kJobCost + (tiles - 1) * kUnits + last_units<TILE>(keys, tiles)) * a.Hkv * a.n_rt;
}

__device__ __forceinline__ int warp_scan(int x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    return x;
}

// This block's share: its first tile and the position behind its last; false
// where it has none.  Called by whole warps: each counts for itself, a lane a
// run of sequences, which costs no barrier.
template <int TILE>
__device__ __forceinline__ bool find_share(const PagedArgs &a, int lane, Shares &shares, Place &at, int &end)
{
    const int per_lane = (a.B + 31) / 32;
    int mine = 0;
    for (int k = 0; k < per_lane; ++k)
        mine += length_of<TILE>(a, lane * per_lane + k);
    const int incl = a.B == 1 ? __shfl_sync(0xffffffffu, mine, 0) : warp_scan(mine, lane);
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    // every share is a tile long at least, so that each of those that a job is
    // cut into holds one of its tiles
    const int blocks = total > 0 ? min((int)gridDim.x, max(total / kUnits, 1)) : 0;
    if ((int)blockIdx.x >= blocks)
        return false;
    shares.each = total / blocks;
    shares.more = total - shares.each * blocks;
    end = shares.first(blockIdx.x + 1);
    at.pos = shares.first(blockIdx.x);
    // the lane whose run holds the position, the sequence in its run, the job
    const int o = __ffs(__ballot_sync(0xffffffffu, incl > at.pos)) - 1;
    int base = __shfl_sync(0xffffffffu, incl - mine, o);
    at.b = o * per_lane;
    for (int k = 0; per_lane > 1 && k < per_lane; k += 32) {
        const int w = k + lane < per_lane ? length_of<TILE>(a, o * per_lane + k + lane) : 0;
        const int x = warp_scan(w, lane);
        const unsigned in = __ballot_sync(0xffffffffu, base + x > at.pos);
        if (in) {
            const int l = __ffs(in) - 1;
            at.b = o * per_lane + k + l;
            base += __shfl_sync(0xffffffffu, x - w, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, x, 31);
    }
    enter<TILE>(a, at);
    const int length = kJobCost + (at.tiles - 1) * kUnits + last_units<TILE>(at.keys, at.tiles);
    at.hr = (at.pos - base) / length;
    // the first tile whose first unit lies in the share
    const int job = base + at.hr * length + kJobCost;
    at.j = max(at.pos - job + kUnits - 1, 0) / kUnits;
    at.pos = job + at.j * kUnits;
    if (at.j == at.tiles) {
        at.j = at.tiles - 1;
        at.pos -= kUnits;
        const int pos = next_pos<TILE>(at);
        if (pos >= end)
            return false;
        advance<TILE>(a, at, pos);
    }
    return at.pos < end;
}

// Joins the parts of a job that was cut between blocks: block x of this kernel
// the job whose first part lies at the end of block x of the first kernel, if
// there is one, and of its rows kJoinWarps / join_warps, beginning at
// blockIdx.y times that.  join_warps warps join every join_warps-th part of a
// row, then through shared memory.
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) attn_paged_join_kernel(const __grid_constant__ PagedArgs a)
{
    constexpr int W = kJoinWarps, PER = D / 32;
    __shared__ float part[W][D], tops[W], sums[W];
    asm volatile("" ::"l"(a.ws_rec), "l"(a.ws_ml), "l"(a.ws_o), "r"(a.n_rt), "r"(a.R), "r"(a.Sq), "l"(a.out), "l"(a.lse),
                 "l"(a.cache.v_scale), "r"(a.out_bf16), "r"(a.join_warps));
    chain_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pw = a.join_warps, rows = W / pw;
    const int row0 = blockIdx.y * rows, row = row0 + warp / pw;
    const int4 rec = __ldcg(a.ws_rec + blockIdx.x);
    const int first = blockIdx.x, last = rec.w, job = rec.x, n_new = rec.y;
    if (last < 0)
        return;
    const int bh = job / a.n_rt, job_row = (job - bh * a.n_rt) * ROWS;
    // a row of the tile that is a row of the output
    auto there = [&](int i) {
        return i < ROWS && job_row + i < a.R && (a.Sq == 1 || (job_row + i) % a.Sq < n_new);
    };
    const int n = there(row) ? last - first + 1 : 0;
    float top = -INFINITY, sum = 0.f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e)
        o[e] = 0.f;
    constexpr int U = kJoinAhead;
    for (int i0 = warp % pw; i0 < n; i0 += pw * U) {
        float2 ml[U];
        float x[U][PER];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * pw;
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                x[u][e] = 0.f;
            if (i < n) {
                const long long s = (long long)(2 * (first + i) + (i == 0 ? 1 : 0)) * ROWS + row;
                ml[u] = __ldcg(a.ws_ml + s);
                const float *src = a.ws_o + s * D + lane * PER;
                if constexpr (PER == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                    x[u][0] = v.x, x[u][1] = v.y, x[u][2] = v.z, x[u][3] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                    x[u][0] = v.x, x[u][1] = v.y;
                }
            }
        }
        float m = top;
#pragma unroll
        for (int u = 0; u < U; ++u)
            m = fmaxf(m, ml[u].x);
        const float ref = m == -INFINITY ? 0.f : m;
        const float f0 = ex2_approx(top - ref);
        top = m;
        sum *= f0;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            o[e] *= f0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = ex2_approx(ml[u].x - ref);
            sum += f * ml[u].y;
#pragma unroll
            for (int e = 0; e < PER; ++e)
                o[e] += f * x[u][e];
        }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e)
        part[warp][lane * PER + e] = o[e];
    if (lane == 0) {
        tops[warp] = top;
        sums[warp] = sum;
    }
    __syncthreads();
    for (int at = tid; at < rows * D; at += W * 32) {
        const int i = at / D, col = at % D, w0 = i * pw;
        if (!there(row0 + i))
            continue;
        top = -INFINITY;
        for (int w = 0; w < pw; ++w)
            top = fmaxf(top, tops[w0 + w]);
        const float ref = top == -INFINITY ? 0.f : top;
        float x = 0.f;
        sum = 0.f;
        for (int w = 0; w < pw; ++w) {
            const float f = ex2_approx(tops[w0 + w] - ref);
            sum += f * sums[w0 + w];
            x += f * part[w0 + w][col];
        }
        const long long at_row = (long long)bh * a.R + job_row + row0 + i;
        x *= sum == 0.f ? 0.f : (a.cache.v_scale ? a.cache.v_scale[bh % a.Hkv] : 1.f) / sum;
        if (a.out_bf16)
            ((__nv_bfloat16 *)a.out)[at_row * D + col] = __float2bfloat16_rn(x);
        else
            ((float *)a.out)[at_row * D + col] = x;
        if (col == 0)
            a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// How many tiles a call may have, a job's cost included.
template <int ROWS, int TILE>
int count_tiles(PagedArgs &a, long long *most, char *msg, size_t msg_len)
{
    a.n_rt = (a.R + ROWS - 1) / ROWS;
    const long long keys = (long long)a.cache.max_pages * a.cache.page_size;
    const long long jobs = (long long)a.B * a.Hkv * a.n_rt;
    static_assert(kJobCost <= 2 * kUnits, "a job's cost counts as two tiles below");
    *most = ((keys + TILE - 1) / TILE + 2) * jobs;
    if (*most > 0x7fffffffLL / kUnits) {
        snprintf(msg, msg_len, "too many key tiles for one call (%lld)", *most);
        return MERCURY_EINVAL;
    }
    return MERCURY_OK;
}

// The first kernel, and the second one where a job may have been cut.
// min_regs: registers a thread that the first one's split counts on.
template <int D, int ROWS, int TILE>
int launch_split(PagedArgs &a, long long most, void (*kernel)(PagedArgs), int smem, int threads, int min_regs,
                 cudaStream_t stream, char *msg, size_t msg_len)
{
    const long long keys = (long long)a.cache.max_pages * a.cache.page_size;
    const long long jobs = (long long)a.B * a.Hkv * a.n_rt;
    KernelInfo ki;
    int rc = prepare_kernel((const void *)kernel, smem, &ki, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    if (ki.regs < min_regs) {
        // the register increase would wait for registers that do not exist
        snprintf(msg, msg_len, "paged attention kernel built with %d registers a thread, needs %d", ki.regs, min_regs);
        return MERCURY_ECUDA;
    }
    // What a call of this shape class with longer sequences needs is made now
    // too, so that it may be captured.
    auto *join = attn_paged_join_kernel<D, ROWS>;
    KernelInfo ji;
    rc = prepare_kernel((const void *)join, 0, &ji, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    cudaMemPool_t pool;
    rc = device_scratch_pool(&pool);
    if (rc != MERCURY_OK)
        return rc;
    // a block per SM, and none that could not get a tile
    const unsigned grid = (unsigned)(most < ki.sms ? most : ki.sms);
    // a job that fits into one tile is never cut: no parts, nothing to join
    const bool split = keys > TILE;
    void *ws = nullptr;
    if (split) {
        const size_t rows = (size_t)2 * grid * ROWS;
        const size_t o_bytes = rows * D * sizeof(float), ml_bytes = rows * sizeof(float2);
        const cudaError_t e = cudaMallocFromPoolAsync(&ws, o_bytes + ml_bytes + grid * sizeof(int4), pool, stream);
        if (e != cudaSuccess) {
            snprintf(msg, msg_len, "paged attention scratch: %s", cudaGetErrorString(e));
            return MERCURY_ECUDA;
        }
        a.ws_o = (float *)ws;
        a.ws_ml = (float2 *)((char *)ws + o_bytes);
        a.ws_rec = (int4 *)((char *)ws + o_bytes + ml_bytes);
    }
    cudaError_t e = launch_chained(kernel, dim3(grid), threads, smem, stream, a);
    if (e == cudaSuccess && split) {
        // As many warps for a row as take its parts in one look, where the
        // jobs are alike; four at least, for jobs that are much longer than
        // the others.  (8 sequences of 16 rows, 64 jobs: 33.4 us, with all
        // eight warps 35.0, since twice the blocks take turns; with two 33.1,
        // but 73.7 instead of 73.0 in the 8-bit case above.)
        const long long parts = grid / jobs + 1;
        for (a.join_warps = 4; a.join_warps < kJoinWarps && a.join_warps * kJoinAhead < parts;)
            a.join_warps *= 2;
        const int rows = kJoinWarps / a.join_warps, used = ROWS < a.R ? ROWS : a.R;
        e = launch_chained(join, dim3(grid, (used + rows - 1) / rows), kJoinWarps * 32, 0,
                           stream, a);
    }
    rc = MERCURY_OK;
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "paged attention launch: %s", cudaGetErrorString(e));
        rc = MERCURY_ECUDA;
    }
    if (ws) {
        e = cudaFreeAsync(ws, stream);
        if (rc == MERCURY_OK && e != cudaSuccess) {
            snprintf(msg, msg_len, "cudaFreeAsync: %s", cudaGetErrorString(e));
            rc = MERCURY_ECUDA;
        }
    }
    return rc;
}

// A call's arguments but for the launch's own.
inline PagedArgs paged_args(const void *q, const Strides &qs, const mercury_paged_cache &cache, const int *seq_lens,
                            const int *new_lens, int B, int Hq, int Sq, int causal, void *out, float *lse, int out_bf16,
                            unsigned long long wait_ns, int fault)
{
    PagedArgs a = {};
    a.wait_ns = wait_ns;
    a.fault = fault;
    a.q = (const __nv_bfloat16 *)q;
    a.qs = qs;
    a.cache = make_view(cache);
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.out = out;
    a.lse = lse;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = cache.Hkv;
    a.G = Hq / cache.Hkv;
    a.Sq = Sq;
    a.R = a.G * Sq;
    a.causal = causal;
    a.out_bf16 = out_bf16;
    a.scale_log2 = kLog2e / sqrtf((float)cache.d);
    return a;
}

}  // namespace
}  // namespace mercury
