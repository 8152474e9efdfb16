// attn_paged.cu -- attention of one new token (or a few) of every sequence
// over a paged cache, split over the cache's length and joined.
//
// For row (b, query head, token i):  x_k = q.k / sqrt(d) over the keys that
// the row sees,  LSE = ln sum_k exp(x_k),  O = sum_k exp(x_k - LSE) v_k,  in
// one pass over the keys with a running maximum and sum.
//
// What bounds it: each key and value is read once for G * Sq query rows, about
// G * Sq operations a byte, so the cache's bytes do, far below what the matrix
// units could take.  The layout follows from that:
//   * a job is one (sequence, KV head, row tile); its keys are cut into tiles,
//     and all tiles of all jobs, in order, are dealt to one block per SM in
//     equal contiguous shares, counted on the device from seq_lens.  A ragged
//     batch is as balanced as an even one, and the host need not know the
//     lengths.  A block writes the jobs it holds whole; of a job cut at a
//     share's end it leaves the unnormalised partial sums, maximum and sum
//     (at most two per block), which a second kernel joins by the exact
//     log-sum-exp rule.  That kernel is resident before the first one ends.
//   * within a block every warp takes its own keys of the tile through its own
//     ring of asynchronous copies and never waits for another warp before the
//     end of a job; rows are looked up in the block table key by key, one tile
//     ahead, so any page size will do and no page has to end with a tile.
//   * both products run on warp-level matrix instructions: the rows of one KV
//     head fill at most 8 to 32 rows of a tile, and the operands come straight
//     from the copied tile.  P goes in as two 16-bit terms (value and
//     remainder), which holds O to 32-bit outputs; with at most 8 rows the
//     remainder rides in the tile's idle half and costs nothing.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"

namespace mercury {

// Error word of this file's kernels: kPagedErrBounds = a length or page
// outside the table or the cache; the first site (0x901 seq_lens, 0x902
// new_lens, 0x903 page).
__device__ unsigned int g_paged_err_word = 0;
__device__ unsigned int g_paged_err_site = 0;

namespace {

constexpr int kJoinThreads = 256;

struct PagedArgs {
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
    int records;    // blocks of the first kernel, for the join kernel
    int tiled;      // pages hold whole runs of 16 keys
    float scale_log2;
};

template <int D, bool FP8, int MT, int W, int CPS>
struct Cfg {
    static constexpr int kWarps = W, kThreads = W * 32;
    static constexpr int kRowB = D * (FP8 ? 1 : 2);        // bytes of one key
    static constexpr int kKeys = kRowB == 256 ? 16 : 32;   // keys of a warp's tile
    static constexpr int kTile = kKeys * kWarps;           // keys of a block's tile
    static constexpr int kPart = kKeys * kRowB;            // bytes of a warp's K (or V) tile
    static constexpr int kStage = 2 * kPart;
    static constexpr int kStages = (232448 / CPS - 1024 - kWarps * (MT == 0 ? 8 : 16 * MT) * 8) / (kWarps * kStage);
    static constexpr int kMt = MT == 0 ? 1 : MT;           // 16-row tiles
    static constexpr int kRows = MT == 0 ? 8 : 16 * MT;
    static constexpr int kPassRows = MT == 0 ? 8 : 16;     // rows reduced at a time
    static constexpr int kSmem = kWarps * kStages * kStage + kWarps * kRows * 8;
    static_assert(kPassRows * D * 4 <= kStage, "a warp's partial rows fit into one of its stages");
};

__device__ __noinline__ void record_bounds(unsigned int site)
{
    atomicOr(&g_paged_err_word, kPagedErrBounds);
    atomicCAS(&g_paged_err_site, 0u, site);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 bytes global -> shared; zeros where !valid (the source is not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8); bf16 operands, or fp16 for an
// 8-bit cache.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
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

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// p as the sum of two 16-bit terms: the nearest, and the nearest to what it
// leaves (2^-18 of p at most in bf16, far less in fp16).
template <bool F16>
__device__ __forceinline__ void split2(float p0, float p1, uint32_t &hi, uint32_t &lo)
{
    if constexpr (F16) {
        hi = pack_f16(p0, p1);
        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        lo = pack_f16(p0 - h.x, p1 - h.y);
    } else {
        hi = pack_bf16(p0, p1);
        lo = pack_bf16(p0 - bf16_lo(hi), p1 - bf16_hi(hi));
    }
}

// 16-byte chunk c of key row r in a copied tile: permuted within 128 bytes so
// that the eight rows of a matrix load hit eight different bank groups.  The
// permutation is an exclusive or with bits of the row, so from a chunk's
// address those of others follow by an exclusive or with a constant.
template <int ROWB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c)
{
    if constexpr (ROWB >= 128)
        return r * ROWB + ((c ^ (r & 7)) << 4);
    else
        return r * ROWB + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ int keys_of(const PagedArgs &a, int b)
{
    const int most = a.cache.max_pages * a.cache.page_size;
    return min(max(__ldg(a.seq_lens + b), 0), most);
}

__device__ __forceinline__ int new_of(const PagedArgs &a, int b)
{
    return a.new_lens ? min(max(__ldg(a.new_lens + b), 0), a.Sq) : a.Sq;
}

// Positions.  All tiles of all jobs lie on one line, on which a job takes
// kJobCost positions without a tile before its tiles: what beginning and
// ending a job costs a block, in tiles, so that a share with many short jobs
// is not longer than one with a few long ones.
constexpr int kJobCost = 1;

// A tile on that line.
struct Place {
    int pos;          // its position
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

// Whether the share that ends at `end` has another tile behind p.
__device__ __forceinline__ bool has_next(const Place &p, int end)
{
    return p.pos + 1 + (p.j + 1 < p.tiles ? 0 : kJobCost) < end;
}

// That tile.
template <int TILE>
__device__ __forceinline__ void advance(const PagedArgs &a, Place &p)
{
    ++p.pos;
    if (++p.j < p.tiles)
        return;
    p.pos += kJobCost;
    p.j = 0;
    if (++p.hr < a.Hkv * a.n_rt)
        return;
    p.hr = 0;
    do {
        ++p.b;  // there is one: the position lies before the end
        enter<TILE>(a, p);
    } while (p.tiles == 0);
}

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
    const int tiles = tiles_of<TILE>(keys_of(a, b), new_of(a, b));
    return tiles == 0 ? 0 : (tiles + kJobCost) * a.Hkv * a.n_rt;
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

template <int D, bool FP8, int MT, int W, int CPS>
__global__ void __launch_bounds__(W * 32, CPS) attn_paged_kernel(const __grid_constant__ PagedArgs a)
{
    using C = Cfg<D, FP8, MT, W, CPS>;
    constexpr int kWarps = W, kThreads = W * 32;
    constexpr int ROWB = C::kRowB, KEYS = C::kKeys, TILE = C::kTile, NS = C::kStages, NT = KEYS / 8;
    constexpr int KK = D / 16, DN = D / 8;  // k-steps of Q.K, 8-column tiles of O
    extern __shared__ __align__(1024) char smem[];
    float *red_m = reinterpret_cast<float *>(smem + kWarps * NS * C::kStage);
    float *red_l = red_m + kWarps * C::kRows;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    chain_wait();

    // ---- this block's share.  Every warp counts for itself, each lane a run of
    // sequences, which costs no barrier.
    const int per_lane = (a.B + 31) / 32;
    int mine = 0;
    for (int k = 0; k < per_lane; ++k)
        mine += length_of<TILE>(a, lane * per_lane + k);
    const int incl = warp_scan(mine, lane);
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (blockIdx.x == 0)
        for (int b = tid; b < a.B; b += kThreads) {
            if (__ldg(a.seq_lens + b) != keys_of(a, b))
                record_bounds(0x901);
            if (a.new_lens && __ldg(a.new_lens + b) != new_of(a, b))
                record_bounds(0x902);
        }
    // every working block gets a position at least, so that the blocks that
    // share a job are neighbours
    const int blocks = min((int)gridDim.x, total);
    if (a.ws_rec && tid == 0)
        a.ws_rec[blockIdx.x] = make_int4(0, 0, 0, -1);
    if ((int)blockIdx.x >= blocks)
        return;
    const Shares shares = {total / blocks, total % blocks};
    const int end = shares.first(blockIdx.x + 1);
    Place at;
    at.pos = shares.first(blockIdx.x);
    {
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
        const int off = at.pos - base, job = off / (at.tiles + kJobCost);
        at.j = off - job * (at.tiles + kJobCost) - kJobCost;
        at.hr = job;
        if (at.j < 0) {  // the share begins between two jobs
            at.pos -= at.j;
            at.j = 0;
        }
        if (at.pos >= end)
            return;
    }

    // ---- the ring of copied tiles: this warp's part of each block tile
    char *const ring = smem + warp * (NS * C::kStage);
    const uint32_t ring_u = smem_addr(ring);
    constexpr int CPR = ROWB / 16, RPP = 32 / CPR;  // chunks of a row, rows copied at a time
    const int my_row = lane / CPR, my_chunk = lane % CPR;
    Place ahead = at;
    bool more = true;  // `ahead` is a tile of this share
    // What was looked up for a copy: how many of the warp's keys exist, their
    // head, and the page and row in it of each run of 16 keys, or where pages
    // do not hold whole runs of 16, of this lane's key.  Two tiles are looked
    // up ahead of the copies: an entry may come from memory, behind the copies
    // in flight.
    constexpr int RUNS = KEYS / 16;
    struct Look {
        int n, h, page[RUNS], row[RUNS];
    };
    Look look = {}, look2 = {};
    auto look_up = [&](Look &l) {
        l.n = 0;
        if (!more)
            return;
        const int key0 = (ahead.j * kWarps + warp) * KEYS;
        l.n = min(ahead.keys - key0, KEYS);
        l.h = a.n_rt == 1 ? ahead.hr : ahead.hr / a.n_rt;
        const int *entries = a.cache.table + ahead.b * a.cache.table_stride;
#pragma unroll
        for (int u = 0; u < RUNS; ++u) {
            const int key = key0 + (a.tiled ? u * 16 : lane % KEYS);
            l.row[u] = -1;
            if (key < ahead.keys) {
                const int pg = page_of(a.cache, key);
                l.row[u] = key - pg * a.cache.page_size;
                l.page[u] = __ldg(entries + pg);
            }
        }
        more = has_next(ahead, end);
        if (more)
            advance<TILE>(a, ahead);
    };
    // byte offset of a row of a page; -1, and a report, for a page that is none
    auto offset_of = [&](int page, int row) {
        if (page >= 0 && page < a.cache.num_pages)
            return (page * a.cache.page_stride + ((long long)look.h * a.cache.page_size + row) * D) * (FP8 ? 1 : 2);
        record_bounds(0x903);
        return -1LL;
    };
    const uint32_t copy_to = ring_u + chunk_at<ROWB>(my_row, my_chunk);
    auto copy_tile = [&](int stage) {
        if (look.n > 0) {
            const uint32_t base = copy_to + stage * C::kStage;
            // row i * RPP + my_row: the same permutation but for these bits
            auto to = [&](int i) { return (base ^ (ROWB >= 128 ? ((i * RPP) & 7) << 4 : 0)) + i * 512; };
            if (a.tiled) {
#pragma unroll
                for (int u = 0; u < RUNS; ++u) {
                    const long long off = look.row[u] >= 0 ? offset_of(look.page[u], look.row[u]) : -1;
                    const long long from = max(off, 0LL) + lane * 16;
                    const char *ks = a.cache.k + from, *vs = a.cache.v + from;
                    constexpr int N = 16 / RPP;
                    if (off >= 0 && look.n >= u * 16 + 16) {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            copy16(to(u * N + i), ks + i * 512);
                            copy16(to(u * N + i) + C::kPart, vs + i * 512);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const bool ok = off >= 0 && u * 16 + i * RPP + my_row < look.n;
                            copy16(to(u * N + i), ks + i * 512, ok);
                            copy16(to(u * N + i) + C::kPart, vs + i * 512, ok);
                        }
                    }
                }
            } else {
                const long long off = look.row[0] >= 0 ? offset_of(look.page[0], look.row[0]) : -1;
#pragma unroll
                for (int i = 0; i < KEYS / RPP; ++i) {
                    const long long o = __shfl_sync(0xffffffffu, off, i * RPP + my_row);
                    const long long from = max(o, 0LL) + my_chunk * 16;
                    copy16(to(i), a.cache.k + from, o >= 0);
                    copy16(to(i) + C::kPart, a.cache.v + from, o >= 0);
                }
            }
        }
        copy_commit();
        look = look2;
        look_up(look2);
    };
    uint32_t qf[C::kMt][KK][MT == 0 ? 2 : 4];
    int h_kv, row0, n_new;  // of the current job: KV head, first row, new tokens
    auto load_q = [&]() {
        h_kv = a.n_rt == 1 ? at.hr : at.hr / a.n_rt;
        row0 = (at.hr - h_kv * a.n_rt) * C::kRows;
        n_new = new_of(a, at.b);
#pragma unroll
        for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
            for (int hf = 0; hf < (MT == 0 ? 1 : 2); ++hf) {
                const int r = row0 + mt * 16 + g + hf * 8;
                const int head = a.Sq == 1 ? r : r / a.Sq, s = r - head * a.Sq;
                const __nv_bfloat16 *src = a.q + at.b * a.qs.b + (h_kv * a.G + head) * a.qs.h + s * a.qs.s;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t x = 0, y = 0;
                    if (r < a.R) {
                        if (FP8) {
                            const uint2 w = *reinterpret_cast<const uint2 *>(src + kk * 16 + 4 * t);
                            x = w.x;
                            y = w.y;
                        } else {
                            x = *reinterpret_cast<const uint32_t *>(src + kk * 16 + 2 * t);
                            y = *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8 + 2 * t);
                        }
                    }
                    qf[mt][kk][hf] = x;
                    qf[mt][kk][MT == 0 ? 1 : 2 + hf] = y;
                }
            }
    };
    load_q();
    look_up(look);
    look_up(look2);
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i)
        copy_tile(i);

    // ---- the tiles
    float acc[C::kMt][DN][4];
    float m_run[C::kMt][2], l_run[C::kMt][2], s_mul[C::kMt][2];
    int lim[C::kMt][2];  // keys that each of this thread's rows sees
    bool fresh = true;  // the tile is the first of its job in this share
    int first_j = at.j;

    constexpr int TPR = (kThreads >= 256 ? 256 : kThreads >= 128 ? 128 : kThreads >= 64 ? 64 : 32) / C::kPassRows;
    constexpr int CP = D / TPR;  // columns of a thread, TPR threads a row, when rows are joined and written
    const int my_line = tid / TPR, col0 = (tid % TPR) * CP;
    // The finished row r of the current job from its maximum, sum and sums.
    auto write_row = [&](int r, float top, float sum, const float (&o)[CP]) {
        if (a.Sq > 1 && r % a.Sq >= n_new)
            return;
        const float f = sum == 0.f ? 0.f : (FP8 ? __ldg(a.cache.v_scale + h_kv) : 1.f) / sum;
        const long long at_row = ((long long)at.b * a.Hkv + h_kv) * a.R + r;
#pragma unroll
        for (int e = 0; e < CP; e += 2) {
            if (a.out_bf16)
                *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.out + at_row * D + col0 + e) =
                    pack_bf16(o[e] * f, o[e + 1] * f);
            else
                *reinterpret_cast<float2 *>((float *)a.out + at_row * D + col0 + e) = make_float2(o[e] * f, o[e + 1] * f);
        }
        if (col0 == 0)
            a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };
    // where the matrix loads of this lane begin in a tile (see the loops)
    const uint32_t k_lane = ring_u + (FP8 ? chunk_at<ROWB>(lane, 0)
                                          : chunk_at<ROWB>((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1));
    const uint32_t v_lane = ring_u + C::kPart + (FP8 ? chunk_at<ROWB>(lane, 0)
                                                     : chunk_at<ROWB>(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4));
    int stage = NS - 1;
    for (;;) {
        const int refill = stage;  // the stage that the last tile left
        stage = stage == NS - 1 ? 0 : stage + 1;
        copy_wait<NS - 2>();
        __syncwarp();
        copy_tile(refill);

        if (fresh) {
            fresh = false;
            first_j = at.j;
            // a factor of at least 2^-120, so that a masked score stays -inf
            // under it; a scale's sign goes to the queries
            float kmul = a.scale_log2;
            uint32_t flip = 0;
            if (FP8) {
                kmul *= __ldg(a.cache.k_scale + h_kv);
                flip = kmul < 0.f ? 0x80008000u : 0u;
                kmul = fabsf(kmul);
            }
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    m_run[mt][hf] = -INFINITY;
                    l_run[mt][hf] = 0.f;
                    const int s = (row0 + mt * 16 + g + hf * 8) % a.Sq;
                    lim[mt][hf] = a.causal ? at.keys - n_new + min(s, n_new - 1) + 1 : at.keys;
                    s_mul[mt][hf] = kmul;
                    if (MT == 0 && hf == 1)
                        continue;
                    if (FP8) {
                        // e4m3 keys widen exactly to fp16, so the queries are
                        // taken to fp16 too: scaled by a power of two that
                        // brings the row's largest element to [2^14, 2^15),
                        // their 8 bits fit exactly down to 2^-28 of it
                        float top = 0.f;
#pragma unroll
                        for (int kk = 0; kk < KK; ++kk) {
                            const uint32_t x = qf[mt][kk][hf], y = qf[mt][kk][MT == 0 ? 1 : 2 + hf];
                            top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(x)), fabsf(bf16_hi(x))),
                                                   fmaxf(fabsf(bf16_lo(y)), fabsf(bf16_hi(y)))));
                        }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        // exponent of 2^(14 - e), kept where both it and its inverse are normal
                        int up = 14 + 127 - (int)(__float_as_uint(top) >> 23);
                        up = min(max(up, -110), 110);
                        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
                        const float mul = kmul * __uint_as_float((uint32_t)(127 - up) << 23);
                        s_mul[mt][hf] = mul < 7.5e-37f ? 7.5e-37f : mul;
#pragma unroll
                        for (int kk = 0; kk < KK; ++kk) {
                            uint32_t &x = qf[mt][kk][hf], &y = qf[mt][kk][MT == 0 ? 1 : 2 + hf];
                            x = pack_f16(bf16_lo(x) * f, bf16_hi(x) * f) ^ flip;
                            y = pack_f16(bf16_lo(y) * f, bf16_hi(y) * f) ^ flip;
                        }
                    }
                }
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int n = 0; n < DN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[mt][n][e] = 0.f;
        }

        const int kb = (at.j * kWarps + warp) * KEYS;
        if (kb < at.keys) {
            const uint32_t k_u = k_lane + stage * C::kStage, v_u = v_lane + stage * C::kStage;
            // ---- S = Q K^T
            float sc[C::kMt][NT][4];
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[mt][n][e] = 0.f;
            if constexpr (!FP8) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        // keys n*8 .. +15, elements kk*16 .. +15
                        uint32_t f[4];
                        ldsm_x4(f, (k_u ^ ((kk & 3) << 5)) + (kk >> 2) * 128 + n * 8 * ROWB);
#pragma unroll
                        for (int mt = 0; mt < C::kMt; ++mt) {
                            const uint32_t a1 = MT == 0 ? 0u : qf[mt][kk][1], a3 = MT == 0 ? 0u : qf[mt][kk][MT == 0 ? 1 : 3];
                            const uint32_t a2 = qf[mt][kk][MT == 0 ? 1 : 2];
                            mma<false>(sc[mt][n], qf[mt][kk][0], a1, a2, a3, f[0], f[1]);
                            mma<false>(sc[mt][n + 1], qf[mt][kk][0], a1, a2, a3, f[2], f[3]);
                        }
                    }
            } else {
                // A matrix load gives each thread four neighbouring elements of
                // a key; the first two stand for columns 2t, 2t+1 of the
                // product's inner axis and the last two for 2t+8, 2t+9, and
                // the queries were loaded in the same order.
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t f[4];
                    ldsm_x4(f, k_u ^ (kk << 4));
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t b0 = e4m3_to_f16(f[n]), b1 = e4m3_to_f16(f[n] >> 16);
#pragma unroll
                        for (int mt = 0; mt < C::kMt; ++mt) {
                            const uint32_t a1 = MT == 0 ? 0u : qf[mt][kk][1], a3 = MT == 0 ? 0u : qf[mt][kk][MT == 0 ? 1 : 3];
                            mma<true>(sc[mt][n], qf[mt][kk][0], a1, qf[mt][kk][MT == 0 ? 1 : 2], a3, b0, b1);
                        }
                    }
                }
            }
            // ---- running maximum and sum; the masked keys of a row count as -inf
            const int seen_by_all = a.causal ? at.keys - n_new + 1 : at.keys;
            const bool edge = kb + KEYS > seen_by_all;
            if (edge) {
#pragma unroll
                for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (kb + n * 8 + t * 2 + (e & 1) >= lim[mt][e >> 1])
                                sc[mt][n][e] = -INFINITY;
            }
            // The maximum moves only when a score exceeds it by 2^8: sum and O
            // share whatever reference the terms were taken with, and the
            // reduction and the rescaling stay off the common path.
            bool grow = false;
            float top[C::kMt][2];
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int hf = 0; hf < (MT == 0 ? 1 : 2); ++hf) {
                    float x = fmaxf(sc[mt][0][hf * 2], sc[mt][0][hf * 2 + 1]);
#pragma unroll
                    for (int n = 1; n < NT; ++n)
                        x = fmaxf(x, fmaxf(sc[mt][n][hf * 2], sc[mt][n][hf * 2 + 1]));
                    top[mt][hf] = x * s_mul[mt][hf];
                    grow |= top[mt][hf] > m_run[mt][hf] + 8.f;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                    for (int hf = 0; hf < (MT == 0 ? 1 : 2); ++hf) {
                        float x = top[mt][hf];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        x = fmaxf(x, m_run[mt][hf]);
                        const float f = x == -INFINITY ? 1.f : ex2(m_run[mt][hf] - x);
                        m_run[mt][hf] = x;
                        l_run[mt][hf] *= f;
#pragma unroll
                        for (int n = 0; n < DN; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                acc[mt][n][hf * 2 + e] *= f;
                                if (MT == 0)
                                    acc[mt][n][2 + e] *= f;
                            }
                    }
            }
            uint32_t p_hi[C::kMt][NT][2], p_lo[C::kMt][NT][2];
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int hf = 0; hf < (MT == 0 ? 1 : 2); ++hf) {
                    const float ref = m_run[mt][hf] == -INFINITY ? 0.f : -m_run[mt][hf];
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float p0 = ex2(fmaf(sc[mt][n][hf * 2], s_mul[mt][hf], ref));
                        const float p1 = ex2(fmaf(sc[mt][n][hf * 2 + 1], s_mul[mt][hf], ref));
                        sum += p0 + p1;
                        split2<FP8>(p0, p1, p_hi[mt][n][hf], p_lo[mt][n][hf]);
                    }
                    l_run[mt][hf] += sum;
                }
            // ---- O += P V
            auto add_pv = [&](float (&d)[4], int mt, int n, uint32_t b0, uint32_t b1) {
                if constexpr (MT == 0) {
                    mma<FP8>(d, p_hi[mt][n][0], p_lo[mt][n][0], p_hi[mt][n + 1][0], p_lo[mt][n + 1][0], b0, b1);
                } else {
                    mma<FP8>(d, p_hi[mt][n][0], p_hi[mt][n][1], p_hi[mt][n + 1][0], p_hi[mt][n + 1][1], b0, b1);
                    mma<FP8>(d, p_lo[mt][n][0], p_lo[mt][n][1], p_lo[mt][n + 1][0], p_lo[mt][n + 1][1], b0, b1);
                }
            };
            // every (two 8-column tiles of O, 16 keys) once: `use` gets the
            // m tile, the column tile, the key tile and the operand
            auto each_v = [&](auto &&use) {
                if constexpr (!FP8) {
#pragma unroll
                    for (int n = 0; n < NT; n += 2)
#pragma unroll
                        for (int c = 0; c < DN; c += 2) {
                            uint32_t f[4];
                            ldsm_x4_t(f, (v_u ^ (((c >> 1) & 3) << 5)) + (c >> 3) * 128 + n * 8 * ROWB);
                            use(c, n, f[0], f[1]);
                            use(c + 1, n, f[2], f[3]);
                        }
                } else {
                    // the transposed load pairs neighbouring elements of a key
                    // in each half: the low bytes of both halves make the
                    // even columns' operand, the high bytes the odd ones'
#pragma unroll
                    for (int c = 0; c < DN; c += 2) {
                        uint32_t f[4];
                        ldsm_x4_t(f, v_u ^ ((c >> 1) << 4));
#pragma unroll
                        for (int n = 0; n < 4; n += 2) {
                            const uint32_t x = __byte_perm(f[n], 0, 0x3120), y = __byte_perm(f[n + 1], 0, 0x3120);
                            use(c, n, e4m3_to_f16(x), e4m3_to_f16(y));
                            use(c + 1, n, e4m3_to_f16(x >> 16), e4m3_to_f16(y >> 16));
                        }
                    }
                }
            };
            // A key that only some rows see still meets the others' products,
            // as 0 * v: harmless unless v is infinite or NaN.
            bool poison = false;
            if (edge && a.causal && n_new > 1) {
                const int r0 = max(seen_by_all - kb, 0), r1 = min(at.keys - kb, KEYS);
                for (int r = r0; r < r1; ++r)
                    for (int w = lane; w < ROWB / 4; w += 32) {
                        const uint32_t x = *reinterpret_cast<const uint32_t *>(ring + stage * C::kStage + C::kPart + r * ROWB + w * 4);
                        poison |= FP8 ? ((x & 0x7fu) == 0x7fu || (x & 0x7f00u) == 0x7f00u ||
                                         (x & 0x7f0000u) == 0x7f0000u || (x & 0x7f000000u) == 0x7f000000u)
                                      : ((x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u);
                    }
                poison = __any_sync(0xffffffffu, poison);
            }
            if (!poison) {
                each_v([&](int c, int n, uint32_t b0, uint32_t b1) {
#pragma unroll
                    for (int mt = 0; mt < C::kMt; ++mt)
                        add_pv(acc[mt][c], mt, n, b0, b1);
                });
            } else {
                // token by token, the last first: the keys that token s does
                // not see are zeroed, and only its rows take the product
                for (int s = n_new - 1; s >= 0; --s) {
                    const int seen = at.keys - n_new + s + 1;
                    __syncwarp();
                    for (int r = max(seen - kb, 0); r < KEYS; ++r)
                        for (int w = lane; w < ROWB / 4; w += 32)
                            *reinterpret_cast<uint32_t *>(ring + stage * C::kStage + C::kPart + r * ROWB + w * 4) = 0u;
                    __syncwarp();
                    each_v([&](int c, int n, uint32_t b0, uint32_t b1) {
#pragma unroll
                        for (int mt = 0; mt < C::kMt; ++mt) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            add_pv(d, mt, n, b0, b1);
                            const int r = row0 + mt * 16 + g;
                            const bool own0 = r % a.Sq == s, own1 = MT == 0 ? own0 : (r + 8) % a.Sq == s;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (e < 2 ? own0 : own1)
                                    acc[mt][c][e] += d[e];
                        }
                    });
                }
            }
        }

        // ---- the job's or the share's end: join the warps
        const bool last_tile = at.j == at.tiles - 1;
        const bool on = has_next(at, end);
        if (last_tile || !on) {
            const bool whole = first_j == 0 && last_tile;
            const int slot = 2 * blockIdx.x + (first_j == 0 ? 1 : 0);
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt) {
                if (mt > 0)
                    __syncthreads();
                float *mine = reinterpret_cast<float *>(ring + stage * C::kStage);
                __syncwarp();
#pragma unroll
                for (int hf = 0; hf < (MT == 0 ? 1 : 2); ++hf) {
                    float l = l_run[mt][hf];
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    const int row = g + hf * 8;
                    if (t == 0) {
                        red_m[warp * C::kRows + mt * 16 + row] = m_run[mt][hf];
                        red_l[warp * C::kRows + mt * 16 + row] = l;
                    }
#pragma unroll
                    for (int n = 0; n < DN; n += FP8 ? 2 : 1) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[e] = acc[mt][n][hf * 2 + e] + (MT == 0 ? acc[mt][n][2 + e] : 0.f);
                            if (FP8)
                                x[2 + e] = acc[mt][n + 1][hf * 2 + e] + (MT == 0 ? acc[mt][n + 1][2 + e] : 0.f);
                        }
                        if (FP8) {
                            const int col = n * 8 + t * 4;
                            *reinterpret_cast<float4 *>(mine + row * D + (((col >> 3) ^ (row & 7)) << 3) + (col & 7)) =
                                make_float4(x[0], x[2], x[1], x[3]);
                        } else {
                            *reinterpret_cast<float2 *>(mine + row * D + ((n ^ (row & 7)) << 3) + t * 2) =
                                make_float2(x[0], x[1]);
                        }
                    }
                }
                __syncthreads();
                const int row = my_line, r = row0 + mt * 16 + row;
                if (row < C::kPassRows && r < a.R) {
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        top = fmaxf(top, red_m[w * C::kRows + mt * 16 + row]);
                    const float ref = top == -INFINITY ? 0.f : top;
                    float sum = 0.f, o[CP];
#pragma unroll
                    for (int e = 0; e < CP; ++e)
                        o[e] = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float f = ex2(red_m[w * C::kRows + mt * 16 + row] - ref);
                        sum += f * red_l[w * C::kRows + mt * 16 + row];
                        const float *src =
                            reinterpret_cast<const float *>(smem + w * (NS * C::kStage) + stage * C::kStage) + row * D;
#pragma unroll
                        for (int e = 0; e < CP; e += 2) {
                            const int col = col0 + e;
                            const float2 x = *reinterpret_cast<const float2 *>(src + (((col >> 3) ^ (row & 7)) << 3) + (col & 7));
                            o[e] += f * x.x;
                            o[e + 1] += f * x.y;
                        }
                    }
                    if (whole) {
                        write_row(r, top, sum, o);
                    } else {
                        const long long at_ws = (long long)slot * C::kRows + mt * 16 + row;
#pragma unroll
                        for (int e = 0; e < CP; e += 2)
                            *reinterpret_cast<float2 *>(a.ws_o + at_ws * D + col0 + e) = make_float2(o[e], o[e + 1]);
                        if (col0 == 0)
                            a.ws_ml[at_ws] = make_float2(top, sum);
                    }
                }
            }
            if (first_j == 0 && !last_tile && tid == 0)  // the first part of a cut job: where is its last?
                a.ws_rec[blockIdx.x] = make_int4(at.b * a.Hkv * a.n_rt + at.hr, n_new, 0,
                                                 shares.owner(at.pos - at.j + at.tiles - 1));
            __syncthreads();
            fresh = true;
        }
        if (!on)
            break;
        advance<TILE>(a, at);
        if (fresh)
            load_q();
    }
    copy_wait<0>();
}

// Joins the parts of the jobs that were cut between blocks: blockIdx.y is a row
// of the tile, and each block takes the records of every gridDim.x-th block of
// the first kernel, 32 in one look.  Each warp joins every eighth part of the
// row, then the warps join through shared memory.
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const __grid_constant__ PagedArgs a)
{
    constexpr int W = kJoinThreads / 32, PER = D / 32;
    __shared__ float part[W][D], tops[W], sums[W];
    chain_wait();
    const int row = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int from = blockIdx.x; from < a.records; from += 32 * gridDim.x) {
        const int mine = from + lane * gridDim.x;
        int4 rec = make_int4(0, 0, 0, -1);
        if (mine < a.records)
            rec = __ldcg(a.ws_rec + mine);
        unsigned todo = __ballot_sync(0xffffffffu, rec.w >= 0);
        while (todo) {
            const int l = __ffs(todo) - 1;
            todo &= todo - 1;
            const int first = from + l * gridDim.x, last = __shfl_sync(0xffffffffu, rec.w, l);
            const int job = __shfl_sync(0xffffffffu, rec.x, l), n_new = __shfl_sync(0xffffffffu, rec.y, l);
            const int bh = job / a.n_rt, r = (job - bh * a.n_rt) * ROWS + row;
            if (r >= a.R || (a.Sq > 1 && r % a.Sq >= n_new))
                continue;
            const int n = last - first + 1;
            float top = -INFINITY, sum = 0.f, o[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e)
                o[e] = 0.f;
            constexpr int U = 8;  // parts in flight
            for (int i0 = warp; i0 < n; i0 += W * U) {
                float2 ml[U];
                float x[U][PER];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * W;
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
                const float f0 = ex2(top - ref);
                top = m;
                sum *= f0;
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    o[e] *= f0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float f = ex2(ml[u].x - ref);
                    sum += f * ml[u].y;
#pragma unroll
                    for (int e = 0; e < PER; ++e)
                        o[e] += f * x[u][e];
                }
            }
            __syncthreads();  // the last job's sums have been read
#pragma unroll
            for (int e = 0; e < PER; ++e)
                part[warp][lane * PER + e] = o[e];
            if (lane == 0) {
                tops[warp] = top;
                sums[warp] = sum;
            }
            __syncthreads();
            if (tid >= D)
                continue;
            top = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w)
                top = fmaxf(top, tops[w]);
            const float ref = top == -INFINITY ? 0.f : top;
            float x = 0.f;
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = ex2(tops[w] - ref);
                sum += f * sums[w];
                x += f * part[w][tid];
            }
            const long long at_row = (long long)bh * a.R + r;
            x *= sum == 0.f ? 0.f : (a.cache.v_scale ? __ldg(a.cache.v_scale + bh % a.Hkv) : 1.f) / sum;
            if (a.out_bf16)
                ((__nv_bfloat16 *)a.out)[at_row * D + tid] = __float2bfloat16_rn(x);
            else
                ((float *)a.out)[at_row * D + tid] = x;
            if (tid == 0)
                a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
    }
}

template <int D, bool FP8, int MT, int W, int CPS>
int launch(PagedArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    using C = Cfg<D, FP8, MT, W, CPS>;
    a.n_rt = (a.R + C::kRows - 1) / C::kRows;
    a.tiled = a.cache.page_size % 16 == 0;
    const long long keys = (long long)a.cache.max_pages * a.cache.page_size;
    const long long jobs = (long long)a.B * a.Hkv * a.n_rt;
    const long long most = ((keys + C::kTile - 1) / C::kTile + kJobCost) * jobs;
    if (most > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many key tiles for one call (%lld)", most);
        return MERCURY_EINVAL;
    }
    auto *kernel = attn_paged_kernel<D, FP8, MT, W, CPS>;
    KernelInfo ki;
    int rc = prepare_kernel((const void *)kernel, C::kSmem, &ki, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    // as many blocks as the SMs hold at once, and none that could not get a tile
    const unsigned grid = (unsigned)(most < ki.sms * CPS ? most : ki.sms * CPS);
    a.records = (int)grid;
    // a job that fits into one tile is never cut: no parts, nothing to join
    const bool split = keys > C::kTile;
    void *ws = nullptr;
    if (split) {
        cudaMemPool_t pool;
        rc = device_scratch_pool(&pool);
        if (rc != MERCURY_OK)
            return rc;
        const size_t rows = (size_t)2 * grid * C::kRows;
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
    cudaError_t e = launch_chained(kernel, dim3(grid), C::kThreads, C::kSmem, stream, a);
    if (e == cudaSuccess && split)
        e = launch_chained(attn_paged_join_kernel<D, C::kRows>, dim3(grid < (unsigned)ki.sms ? grid : ki.sms, C::kRows < a.R ? C::kRows : a.R),
                           kJoinThreads, 0, stream, a);
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

template <int D, bool FP8>
int launch_rows(PagedArgs &a, int sms, cudaStream_t stream, char *msg, size_t msg_len)
{
    // Warps a block and blocks an SM, measured at the sizes named.  Eight warps
    // in one block leave the fewest parts to join (one 4K sequence of 8 KV
    // heads: 8.5 us against 9.4 with three blocks of four).  Many short jobs
    // want several blocks, one of which streams while another changes jobs (64
    // sequences of 1 to 2047 tokens, 16 heads of 64: 53 us in one block, 48 in
    // three), and so do 8-bit keys, whose conversions one block does not hide
    // (8 sequences of 20K to 32K: 79 against 75 us).
    const long long jobs = (long long)a.B * a.Hkv;
    if (a.R <= 8) {
        if (jobs >= 2 * sms)
            return launch<D, FP8, 0, 4, 3>(a, stream, msg, msg_len);
        return FP8 ? launch<D, FP8, 0, 4, 2>(a, stream, msg, msg_len) : launch<D, FP8, 0, 8, 1>(a, stream, msg, msg_len);
    }
    if (a.R <= 16)
        return FP8 ? launch<D, FP8, 1, 4, 2>(a, stream, msg, msg_len) : launch<D, FP8, 1, 8, 1>(a, stream, msg, msg_len);
    return launch<D, FP8, 2, 4, 2>(a, stream, msg, msg_len);
}

}  // namespace

int launch_attn_paged(const void *q, const Strides &qs, const mercury_paged_cache &cache, const int *seq_lens,
                      const int *new_lens, int B, int Hq, int Sq, int causal, void *out, float *lse, int out_bf16,
                      cudaStream_t stream, char *msg, size_t msg_len)
{
    PagedArgs a = {};
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
    int sms = 0;
    int rc = device_sm_count(&sms);
    if (rc != MERCURY_OK)
        return rc;
    const bool fp8 = cache.elem == MERCURY_ELEM_E4M3;
    if (!fp8)
        a.cache.v_scale = nullptr;
    if (cache.d == 128)
        return fp8 ? launch_rows<128, true>(a, sms, stream, msg, msg_len) : launch_rows<128, false>(a, sms, stream, msg, msg_len);
    return fp8 ? launch_rows<64, true>(a, sms, stream, msg, msg_len) : launch_rows<64, false>(a, sms, stream, msg, msg_len);
}

int read_and_clear_paged_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    unsigned int zero = 0, w = 0, st = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_paged_err_word, sizeof w);
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbol(&st, g_paged_err_site, sizeof st);
    if (e == cudaSuccess && (w || st)) {
        e = cudaMemcpyToSymbol(g_paged_err_word, &zero, sizeof zero);
        if (e == cudaSuccess)
            e = cudaMemcpyToSymbol(g_paged_err_site, &zero, sizeof zero);
    }
    if (e != cudaSuccess) {
        snprintf(msg, msg_len, "reading the paged attention error word: %s", cudaGetErrorString(e));
        return MERCURY_ECUDA;
    }
    *word = w;
    *site = st;
    return MERCURY_OK;
}

}  // namespace mercury
