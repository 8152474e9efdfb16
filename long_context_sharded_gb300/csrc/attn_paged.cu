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
//     log-sum-exp rule.  Its blocks come up as those of the first leave their
//     SMs, which they fill.
//   * in a block four warps do nothing but look up pages and send tensor
//     copies of whole tiles into a ring of stages, across the ends of jobs, so
//     the memory is kept busy while the other eight change jobs; with copies
//     and look-ups spread over the computing warps these took more of a tile's
//     time (1000 cycles of 2800) than its products.
//   * both products run on warp-level matrix instructions: the rows of one KV
//     head fill 8 to 64 rows of a tile, and the operands come straight from
//     the copied tile.  P goes in as three bf16 terms (two fp16 ones with 8-bit
//     keys), and the matrix unit's sums are kept short, which keeps O as near
//     to 64 bits as a 32-bit softmax; with at most 8 rows two terms share an
//     instruction, whose lower half would idle.
//
// Measured on a GB300, of the measured copy bandwidth (6770 GB/s): 16 sequences
// of 700 to 32K tokens, 64 query and 8 KV heads of 128: 160 us, 101 %; one
// sequence of 128K: 81 us, 98 %; 8 sequences of 20K to 32K with 16 rows a KV
// head: 134 us, 95 %; with 28 rows, where the matrix instructions and the
// additions of their sums bound it, 176 us, 72 %, with 56 rows 313 us, 41 %.
// 8-bit keys and values, 4 rows: 72 us, 89 %, bound by the conversions (64 of a
// warp's 450 instructions a step of 32 keys for each product) and the latency of
// two warps a quarter of an SM; 16 rows 86 us, 74 %, 28 rows 151 us, 42 %, 56
// rows 283 us, 23 %, each row group converting for itself.  One 4K sequence
// takes 8.6 us, of which the start (lengths, pages, the first tile) is 3.5 and
// the second kernel 2.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mercury {

// Error word of this file's kernels: kPagedErrBounds = a length or page
// outside the table or the cache, kErrTimeout = a bounded wait ran out; the
// first site (0x901 seq_lens, 0x902 new_lens, 0x903 page, 0x904 wait).
__device__ unsigned int g_paged_err_word = 0;
__device__ unsigned int g_paged_err_site = 0;

namespace {

constexpr int kWarps = 8;                    // computing warps of a block
constexpr int kCopyWarps = 4;                // and those that copy
constexpr int kThreads = (kWarps + kCopyWarps) * 32;
// Registers a thread after the split (setmaxnreg): the copying warpgroup's go
// to the computing ones.  Their sum may not exceed what the launch provides.
constexpr uint32_t kRegsCopy = 72;
constexpr uint32_t kRegsCompute = 216;
constexpr int kMinLaunchRegs = (int)(kRegsCopy * 128 + kRegsCompute * kWarps * 32 + kThreads - 1) / kThreads;
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

// RG: 16-row groups of a row tile; 0 for a tile of 8 rows.  The computing
// warps are RG row groups times 8 / RG key groups, each with kKeys keys at a
// time; a tile's keys are the same for every RG.
template <int D, bool FP8, int RG>
struct Cfg {
    static constexpr int kRowB = D * (FP8 ? 1 : 2);            // bytes of one key
    static constexpr int kBoxB = kRowB < 128 ? kRowB : 128;    // bytes of a key in one box
    static constexpr int kKeys = kRowB == 256 ? 16 : 32;       // keys of a warp's step
    static constexpr int kTile = kKeys * kWarps;               // keys of a block's tile
    static constexpr int kRg = RG == 0 ? 1 : RG;
    static constexpr int kKg = kWarps / kRg;
    static constexpr int kPart = kTile * kRowB;                // bytes of a tile's keys (or values)
    static constexpr int kStage = 2 * kPart;
    static constexpr int kStages = 196608 / kStage;
    static constexpr int kRows = RG == 0 ? 8 : 16 * RG;
    static constexpr int kWarpRows = RG == 0 ? 8 : 16;
    static constexpr int kRed = kWarps * kWarpRows * 8;        // each warp's maxima and sums
    static constexpr int kRowBytes = kWarps * kWarpRows * D * 4;  // the warps' partial rows
    static constexpr int kCtl = kStages * kStage + kRed + kStages * 16;  // the block's Stop
    static constexpr int kRowsAt = kCtl + 32;
    static constexpr bool kOwnRows = kRowsAt + kRowBytes <= 232448;
    static constexpr int kSmem = kRowsAt + (kOwnRows ? kRowBytes : 0);
    static_assert(kTile % (32 * kCopyWarps) == 0, "whole runs for each copying warp");
    static_assert(kWarps * kWarpRows * D * 4 <= kStage, "the warps' partial rows fit into a stage");
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

// 16 bytes global -> shared; zeros where !valid (the source is not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

// One arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Arrive on a named barrier without waiting.
__device__ __forceinline__ void named_barrier_arrive(uint32_t id, uint32_t nthreads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
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

// 4-D tiled bulk tensor load global -> shared, completion counted in bytes on
// `bar`; c0 (elements) is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2,
                                            int c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
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

// For each element of w, two of bf16 or four of e4m3, that is infinite or NaN
// (whose exponent bits, or all bits but the sign, are ones) its lowest bit.
template <bool FP8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    return FP8 ? ((w & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u : ((w & 0x7f807f80u) + 0x00800080u) >> 15 & 0x00010001u;
}

// A copied tile's keys (or values): boxes of all its keys x kBoxB bytes (128,
// or 64 for heads of 64 bytes), the 16-byte chunks of a row permuted so that
// the eight rows of a matrix load hit eight different bank groups -- the
// layout of a tensor copy with 128- (64-) byte swizzle.  The permutation is an
// exclusive or with bits of the row, so from a chunk's address those of others
// follow by an exclusive or with a constant.
template <int ROWB, int TILE>
__device__ __forceinline__ uint32_t chunk_at(int r, int c)
{
    constexpr int B = ROWB < 128 ? ROWB : 128, CB = B / 16;
    const int x = ROWB >= 128 ? r & 7 : (r >> 1) & 3;
    return c / CB * TILE * B + r * B + (((c % CB) ^ x) << 4);
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

// The copying warps: every tile of the share into the ring, a stage as soon as
// the computing warps have left it.  A tile's boxes (or runs of 32 keys) are
// dealt to the four warps in turn: with pages of 16 keys a tile is 32 tensor
// copies, which took one warp 2200 cycles.
template <int D, bool FP8, int RG>
__device__ __forceinline__ void copy_tiles(const PagedArgs &a, Place at, int end, char *smem, uint64_t *full,
                                           uint64_t *empty, Stop *stop, int warp, int lane)
{
    using C = Cfg<D, FP8, RG>;
    constexpr int ROWB = C::kRowB, TILE = C::kTile, NS = C::kStages, N = TILE / 32 / kCopyWarps;
    constexpr int ES = FP8 ? 1 : 2, CPR = ROWB / 16, RPP = 32 / CPR;  // chunks of a row, rows copied at a time
    // Page entries of the next tile, asked for a tile ahead: with tensor
    // copies lane l's is that of box l * kCopyWarps + warp, else those of key l
    // of this warp's runs.
    int entry[N];
    const int first = (lane * kCopyWarps + warp) * a.box_rows;  // this lane's box
    auto run = [&](int i) { return (i * kCopyWarps + warp) * 32; };
    auto key_of = [&](int i) { return at.j * TILE + (a.box_rows ? first : run(i) + lane); };
    auto look_up = [&]() {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i == 0 || !a.box_rows) && key_of(i) < at.keys)
                entry[i] = a.cache.table[at.b * a.cache.table_stride + page_of(a.cache, key_of(i))];
    };
    look_up();
    int stage = 0;
    uint32_t phase = 1;  // a fresh ring's stages count as left
    int sent = 0;
    while (!(a.fault && warp == 0)) {  // (the test hook: the first of the four sends nothing)
        const int next = next_pos<TILE>(at);
        const bool on = next < end;
        const int h = a.n_rt == 1 ? at.hr : at.hr / a.n_rt;
        char *const part = smem + stage * C::kStage;
        wait_phase(empty + stage, phase, a.wait_ns, stop);
        if (__any_sync(0xffffffffu, stopped(stop)))
            break;
        if (a.box_rows) {
            const int key = key_of(0);
            const int page = entry[0], row = key - page_of(a.cache, key) * a.cache.page_size;
            const bool live = first < TILE && key < at.keys;
            const bool good = live && page >= 0 && page < a.cache.num_pages;
            if (live && !good) {  // such keys count as zeros
                record_bounds(0x903);
                for (int r = first; r < first + a.box_rows; ++r)
                    for (int c = 0; c < CPR; ++c) {
                        const uint32_t to = smem_u32(part) + chunk_at<ROWB, TILE>(r, c);
                        st_shared_v4(to, 0, 0, 0, 0);
                        st_shared_v4(to + C::kPart, 0, 0, 0, 0);
                    }
                fence_proxy_async_smem();
            }
            __syncwarp();  // every lane's zeros stand before lane 0's arrival
            const int boxes = __popc(__ballot_sync(0xffffffffu, good));
            if (lane == 0)
                mbar_arrive_expect_tx(full + stage, boxes * a.box_rows * 2 * ROWB);
            __syncwarp();
            if (good) {
#pragma unroll
                for (int x = 0; x < ROWB / C::kBoxB; ++x) {
                    const uint32_t to = smem_u32(part) + x * TILE * C::kBoxB + first * C::kBoxB;
                    tma_load_4d(to, &a.map_k, smem_u32(full + stage), x * (C::kBoxB / ES), row, h, page);
                    tma_load_4d(to + C::kPart, &a.map_v, smem_u32(full + stage), x * (C::kBoxB / ES), row, h, page);
                }
            }
        } else {
            const int my_row = lane / CPR, my_chunk = lane % CPR;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int key = key_of(i);
                long long off = -1;  // byte offset of this lane's key
                if (key < at.keys) {
                    if (entry[i] >= 0 && entry[i] < a.cache.num_pages)
                        off = (entry[i] * a.cache.page_stride +
                               ((long long)h * a.cache.page_size + key - page_of(a.cache, key) * a.cache.page_size) * D) * ES;
                    else
                        record_bounds(0x903);
                }
#pragma unroll 4
                for (int p = 0; p < CPR; ++p) {
                    const int r = p * RPP + my_row;
                    const long long o = __shfl_sync(0xffffffffu, off, r), from = max(o, 0LL) + my_chunk * 16;
                    const uint32_t to = smem_u32(part) + chunk_at<ROWB, TILE>(run(i) + r, my_chunk);
                    copy16(to, a.cache.k + from, o >= 0);
                    copy16(to + C::kPart, a.cache.v + from, o >= 0);
                }
            }
            copy_arrive(full + stage);
        }
        ++sent;
        if (!on)
            break;
        advance<TILE>(a, at, next);
        look_up();
        if (at.j == 0 && warp == 0) {
            // a new job: its queries into L2 by the time the computing warps
            // get there
            const int h1 = a.n_rt == 1 ? at.hr : at.hr / a.n_rt, row0 = (at.hr - h1 * a.n_rt) * C::kRows;
            for (int r = row0 + lane; r < min(row0 + C::kRows, a.R); r += 32) {
                const int head = a.Sq == 1 ? r : r / a.Sq, s = r - head * a.Sq;
                const __nv_bfloat16 *src = a.q + at.b * a.qs.b + (h1 * a.G + head) * a.qs.h + s * a.qs.s;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
                if (D == 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
            }
        }
        if (++stage == NS) {
            stage = 0;
            phase ^= 1;
        }
    }
    // The block's memory is given up only when nothing is on its way there.
    // Where no wait ran out, the computing warps have seen every tile land.
    if (lane == 0)
        stop->sent[warp] = sent;
    named_barrier_sync(kEndBarrier, kThreads);
    if (!stopped(stop))
        return;
    // Else the tiles that are not known to have landed are the last NS that any
    // of the four sent: tile i goes out only when i - NS has landed in full and
    // been left, and nothing goes out after a stop.  For the same reason this
    // warp owes each of their barriers at most one arrival; with those made up
    // they complete as the copies land.
    int most = 0;
    for (int w = 0; w < kCopyWarps; ++w)
        most = max(most, stop->sent[w]);
    for (int i = sent; i < most; ++i)
        if (!a.box_rows || lane == 0)
            mbar_arrive(full + i % NS);
    for (int i = max(most - NS, 0); i < most; ++i) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(full + i % NS, i / NS & 1) && globaltimer_ns() - t0 <= a.wait_ns)
            ;
    }
}

template <int D, bool FP8, int RG>
__global__ void __launch_bounds__(kThreads, 1) attn_paged_kernel(const __grid_constant__ PagedArgs a)
{
    using C = Cfg<D, FP8, RG>;
    constexpr int ROWB = C::kRowB, KEYS = C::kKeys, TILE = C::kTile, NS = C::kStages, NT = KEYS / 8;
    constexpr int KK = D / 16, DN = D / 8;  // k-steps of Q.K, 8-column tiles of O
    constexpr int BOX = C::kBoxB, BOXES = TILE * BOX;  // bytes from a row to the next, from a box to the next
    extern __shared__ __align__(1024) char smem[];
    float *const red_m = reinterpret_cast<float *>(smem + NS * C::kStage);
    float *const red_l = red_m + kWarps * C::kWarpRows;
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + NS * C::kStage + C::kRed);
    uint64_t *const empty = full + NS;
    Stop *const stop = reinterpret_cast<Stop *>(smem + C::kCtl);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        stop->now = 0;
        for (int i = 0; i < NS; ++i) {
            // a tile has landed: an arrival of each copying warp and the bytes
            // of its tensor copies, or an arrival of each copying lane
            mbar_init(full + i, a.box_rows ? kCopyWarps : kCopyWarps * 32);
            mbar_init(empty + i, kWarps);
        }
        fence_mbar_init();
    }
    // The parameters that the share is found with: fetched while the kernel
    // before this one still runs, where their latency costs nothing.
    asm volatile("" ::"l"(a.seq_lens), "l"(a.new_lens), "r"(a.B), "r"(a.Hkv), "r"(a.n_rt), "r"(a.cache.max_pages),
                 "r"(a.cache.page_size), "l"(a.cache.table), "l"(a.q), "r"(a.Sq), "l"(a.ws_rec), "l"(a.wait_ns));
    if (warp == kWarps && a.box_rows) {
        tma_prefetch_desc(&a.map_k);
        tma_prefetch_desc(&a.map_v);
    }
    chain_wait();
    __syncthreads();
    if (tid == 0 && a.ws_rec)
        a.ws_rec[blockIdx.x] = make_int4(0, 0, 0, -1);
    if (blockIdx.x == 0)
        for (int b = tid; b < a.B; b += kThreads) {
            if (a.seq_lens[b] != keys_of(a, b))
                record_bounds(0x901);
            if (a.new_lens && a.new_lens[b] != new_of(a, b))
                record_bounds(0x902);
        }
    Shares shares;
    Place at;
    int end;
    if (!find_share<TILE>(a, lane, shares, at, end))
        return;
    if (warp >= kWarps) {
        regs_dec<kRegsCopy>();
        copy_tiles<D, FP8, RG>(a, at, end, smem, full, empty, stop, warp - kWarps, lane);
        return;
    }

    // ---- the computing warps
    regs_inc<kRegsCompute>();
    const int g = lane >> 2, t = lane & 3;
    const int kg = warp % C::kKg, rg = warp / C::kKg;  // this warp's keys of a tile, and rows
    uint32_t qf[KK][RG == 0 ? 2 : 4];
    int h_kv, row0, n_new;  // of the current job: KV head, first row, new tokens
    float k_scale = 1.f;
    auto load_q = [&]() {
        h_kv = a.n_rt == 1 ? at.hr : at.hr / a.n_rt;
        row0 = (at.hr - h_kv * a.n_rt) * C::kRows;
        n_new = new_of(a, at.b);
        if (FP8)
            k_scale = a.cache.k_scale[h_kv];
#pragma unroll
        for (int hf = 0; hf < (RG == 0 ? 1 : 2); ++hf) {
            const int r = row0 + rg * 16 + g + hf * 8;
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
                qf[kk][hf] = x;
                qf[kk][RG == 0 ? 1 : 2 + hf] = y;
            }
        }
    };
    load_q();

    // O's sums.  The matrix unit truncates: with O as its accumulator for a
    // whole job, each product lost up to a unit in O's last place, always
    // towards zero (32K keys, 64 rows: 6e-5 of O).  So its own sums, acc, are
    // short, kWindow products from zero, and are added to O's by an ordinary
    // addition.  With more than 8 rows, heads of 128 have no registers for both,
    // nor have heads of 64 with 8-bit keys, whose small terms have sums of their
    // own; those take a step's products at a time (at 20K to 32K keys windows
    // take 9 % longer for 28 rows of 128 and for 16 rows of 64 in 8 bits, but
    // 6 % less for 56 rows of 64 in 16 bits).
    constexpr int TERMS = FP8 ? 2 : 3;
    constexpr int AW = RG == 0 ? 2 : 4;  // sums of this thread in each 8-column tile of O: one row's, or two
    constexpr bool kByStep = RG > 0 && (D == 128 || FP8);
    constexpr int kWindow = 24, kTileProducts = C::kRg * (NT / 2) * (RG == 0 ? 1 : TERMS);
    constexpr int kFlush = kWindow > kTileProducts ? kWindow / kTileProducts : 1;  // tiles of a window
    float sums[DN][AW];
    float acc[kByStep ? 1 : DN][4];  // of eight rows the tile's lower half holds small terms
    constexpr int ACC = FP8 && RG > 0 ? 8 : 4;  // a step's sums: the second terms' behind the first ones'
    int fresh;                       // tiles in acc
    float m_run[2], l_run[2], l_rest[2], s_mul[2];  // l_rest: what the roundings of l_run left out
    auto clear_acc = [&] {
        fresh = 0;
        if constexpr (!kByStep) {
#pragma unroll
            for (int n = 0; n < DN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[n][e] = 0.f;
        }
    };
    auto flush = [&] {
        if constexpr (RG == 0) {
#pragma unroll
            for (int n = 0; n < DN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    sums[n][e] += acc[n][e] + acc[n][2 + e] * (FP8 ? kLow : 1.f);
        } else if constexpr (!kByStep) {
#pragma unroll
            for (int n = 0; n < DN; ++n)
                add_to(sums[n], acc[n], 1.f);
        }
        clear_acc();
    };
    int lim[2];         // keys that each of this thread's rows sees
    // A row of the joined tile belongs to TPR threads, which take its columns
    // in turn, two at a time.
    constexpr int TPR = kWarps * 32 / C::kRows, CP = D / TPR;
    const int my_line = tid / TPR, col0 = tid % TPR * 2;
    // where the matrix loads of this lane begin in a tile (see the loops)
    const uint32_t k_lane = smem_u32(smem) + (FP8 ? chunk_at<ROWB, TILE>(lane, 0)
                                                  : chunk_at<ROWB, TILE>((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1));
    const uint32_t v_lane = smem_u32(smem) + C::kPart +
                            (FP8 ? chunk_at<ROWB, TILE>(lane, 0)
                                 : chunk_at<ROWB, TILE>(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4));
    int stage = 0;
    uint32_t phase = 0;
    // this warp is done with the stage
    auto release = [&] {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(empty + stage);
        if (++stage == NS) {
            stage = 0;
            phase ^= 1;
        }
    };
    for (;;) {
        // ---- a job, or its part in this share: everything that does not need
        // a tile goes before the first wait
        const int first_j = at.j;
        int left = min(at.tiles - at.j, (end - at.pos + kUnits - 1) / kUnits);  // its tiles here
        at.pos += (left - 1) * kUnits;                                          // of the last of them
        // a factor of at least 2^-120, so that a masked score stays -inf
        // under it; a scale's sign goes to the queries
        float kmul = a.scale_log2;
        uint32_t flip = 0;
        if (FP8) {
            kmul *= k_scale;
            flip = kmul < 0.f ? 0x80008000u : 0u;
            kmul = fabsf(kmul);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            m_run[hf] = -INFINITY;
            l_run[hf] = 0.f;
            l_rest[hf] = 0.f;
            const int s = (row0 + rg * 16 + g + hf * 8) % a.Sq;
            lim[hf] = a.causal ? at.keys - n_new + min(s, n_new - 1) + 1 : at.keys;
            s_mul[hf] = kmul;
            if (RG == 0 && hf == 1)
                continue;
            if (FP8) {
                // e4m3 keys widen exactly to fp16, so the queries are
                // taken to fp16 too: scaled by a power of two that brings
                // the row's largest element to [2^14, 2^15), their 8 bits
                // fit exactly down to 2^-28 of it
                float top = 0.f;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    const uint32_t x = qf[kk][hf], y = qf[kk][RG == 0 ? 1 : 2 + hf];
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
                s_mul[hf] = mul < 7.5e-37f ? 7.5e-37f : mul;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t &x = qf[kk][hf], &y = qf[kk][RG == 0 ? 1 : 2 + hf];
                    x = pack_f16(bf16_lo(x) * f, bf16_hi(x) * f) ^ flip;
                    y = pack_f16(bf16_lo(y) * f, bf16_hi(y) * f) ^ flip;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < DN; ++n)
#pragma unroll
            for (int e = 0; e < AW; ++e)
                sums[n][e] = 0.f;
        clear_acc();

        for (;;) {
            wait_phase(full + stage, phase, a.wait_ns, stop);
#pragma unroll 1
            for (int step = kg; step < kWarps; step += C::kKg) {
                const int kb = at.j * TILE + step * KEYS;
                if (kb >= at.keys)
                    break;
                const uint32_t k_u = k_lane + stage * C::kStage + step * KEYS * BOX;
                const uint32_t v_u = v_lane + stage * C::kStage + step * KEYS * BOX;
                // Word w of row r of this step's values.
                auto v_word = [&](int r, int w) {
                    return reinterpret_cast<uint32_t *>(smem + stage * C::kStage + C::kPart + (step * KEYS + r) * BOX +
                                                        w / (BOX / 4) * BOXES) + w % (BOX / 4);
                };
                // A copied box's rows behind the last key may hold anything: their
                // scores are masked, their values must not be infinite or NaN.
                // (Warps of several row groups write the same zeros.)
                // This is the job's last tile, so the fence at the job's end stands
                // between these zeros and the next tensor copy.
                if (kb + KEYS > at.keys) {
                    for (int i = (at.keys - kb) * (ROWB / 16) + lane; i < KEYS * (ROWB / 16); i += 32)
                        st_shared_v4(smem_u32(v_word(i / (ROWB / 16), i % (ROWB / 16) * 4)), 0, 0, 0, 0);
                    __syncwarp();
                }
                // ---- S = Q K^T
                float sc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[n][e] = 0.f;
                if constexpr (!FP8) {
                    // in 2 sums of d/2 products each, added at the end
                    float part[2][NT][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                part[i][n][e] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                        for (int n = 0; n < NT; n += 2) {
                            // keys n*8 .. +15, elements kk*16 .. +15
                            uint32_t f[4];
                            ldsm_x4(f, (k_u ^ ((kk & 3) << 5)) + (kk >> 2) * BOXES + n * 8 * BOX);
                            const uint32_t a1 = RG == 0 ? 0u : qf[kk][1], a3 = RG == 0 ? 0u : qf[kk][RG == 0 ? 1 : 3];
                            const uint32_t a2 = qf[kk][RG == 0 ? 1 : 2];
                            mma<false>(part[kk % 2][n], qf[kk][0], a1, a2, a3, f[0], f[1]);
                            mma<false>(part[kk % 2][n + 1], qf[kk][0], a1, a2, a3, f[2], f[3]);
                        }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < (RG == 0 ? 2 : 4); ++e)
                            sc[n][e] = part[0][n][e] + part[1][n][e];
                } else {
                    // A matrix load gives each thread four neighbouring elements of
                    // a key; the first two stand for columns 2t, 2t+1 of the
                    // product's inner axis and the last two for 2t+8, 2t+9, and
                    // the queries were loaded in the same order.
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        uint32_t f[4];
                        ldsm_x4(f, k_u ^ (kk << 4));
                        const uint32_t a1 = RG == 0 ? 0u : qf[kk][1], a3 = RG == 0 ? 0u : qf[kk][RG == 0 ? 1 : 3];
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            mma<true>(sc[n], qf[kk][0], a1, qf[kk][RG == 0 ? 1 : 2], a3, e4m3_to_f16(f[n]),
                                      e4m3_to_f16(f[n] >> 16));
                    }
                }
                // ---- running maximum and sum; the masked keys of a row count as -inf
                const int seen_by_all = a.causal ? at.keys - n_new + 1 : at.keys;
                const bool edge = kb + KEYS > seen_by_all;
                if (edge) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (kb + n * 8 + t * 2 + (e & 1) >= lim[e >> 1])
                                sc[n][e] = -INFINITY;
                }
                // The maximum moves only when a score exceeds it by 2^kGrow: sum and O
                // share whatever reference the terms were taken with, and the
                // reduction and the rescaling stay off the common path.
                bool grow = false;
                float top[2];
#pragma unroll
                for (int hf = 0; hf < (RG == 0 ? 1 : 2); ++hf) {
                    float x = fmaxf(sc[0][hf * 2], sc[0][hf * 2 + 1]);
#pragma unroll
                    for (int n = 1; n < NT; ++n)
                        x = fmaxf(x, fmaxf(sc[n][hf * 2], sc[n][hf * 2 + 1]));
                    top[hf] = x * s_mul[hf];
                    grow |= top[hf] > m_run[hf] + kGrow<FP8>;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int hf = 0; hf < (RG == 0 ? 1 : 2); ++hf) {
                        float x = top[hf];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        x = fmaxf(x, m_run[hf]);
                        const float f = x == -INFINITY ? 1.f : ex2_approx(m_run[hf] - x);
                        m_run[hf] = x;
                        l_run[hf] *= f;
                        l_rest[hf] *= f;
#pragma unroll
                        for (int n = 0; n < DN; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                sums[n][hf * 2 + e] *= f;
                                if constexpr (!kByStep)
                                    acc[n][hf * 2 + e] *= f;
                                if constexpr (RG == 0)
                                    acc[n][2 + e] *= f;
                            }
                    }
                }
                uint32_t p[NT][2][TERMS];
#pragma unroll
                for (int hf = 0; hf < (RG == 0 ? 1 : 2); ++hf) {
                    const float ref = m_run[hf] == -INFINITY ? 0.f : kUp<FP8> - m_run[hf];
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float p0 = ex2_approx(fmaf(sc[n][hf * 2], s_mul[hf], ref));
                        const float p1 = ex2_approx(fmaf(sc[n][hf * 2 + 1], s_mul[hf], ref));
                        sum += p0 + p1;
                        split<FP8>(p0, p1, p[n][hf]);
                    }
                    // with what is left of earlier roundings: equal weights,
                    // small beside the sum, all round the same way (16K of
                    // them: 2e-5 of the sum)
                    sum += l_rest[hf];
                    const float l = l_run[hf] + sum;
                    l_rest[hf] = sum - (l - l_run[hf]);
                    l_run[hf] = l;
                }
                // ---- O += P V
                auto add_pv = [&](float *d, int n, uint32_t b0, uint32_t b1) {
                    // eight rows take two terms at once, the second in the tile's
                    // lower half, and the third goes there too; else small ones first
                    if constexpr (RG == 0) {
                        mma<FP8>(d, p[n][0][0], p[n][0][1], p[n + 1][0][0], p[n + 1][0][1], b0, b1);
                        if constexpr (TERMS == 3)
                            mma<FP8>(d, 0u, p[n][0][2], 0u, p[n + 1][0][2], b0, b1);
                    } else {
#pragma unroll
                        for (int i = TERMS - 1; i >= 0; --i)
                            mma<FP8>(d + (FP8 ? i * 4 : 0), p[n][0][i], p[n][1][i], p[n + 1][0][i], p[n + 1][1][i], b0, b1);
                    }
                };
                // A key that only some rows see still meets the others' products,
                // as 0 * v: harmless unless v is infinite or NaN.  Such an
                // element is taken as zero, and made NaN in its column of O in
                // the rows that see it (their sum of p's terms times an
                // infinity is one anyway).  In here, not in a second version of
                // the products, whose registers slowed the first (128K keys: by
                // 2 %; 8-bit, 64 rows: by 7).
                if (edge && a.causal && n_new > 1) {
                    const int r0 = max(seen_by_all - kb, 0), r1 = min(at.keys - kb, KEYS);
                    constexpr int WORDS = ROWB / 4, EACH = FP8 ? 4 : 2, BITS = 32 / EACH;
                    auto word = [&](int r, int w) {
                        return reinterpret_cast<uint32_t *>(smem + stage * C::kStage + C::kPart +
                                                            chunk_at<ROWB, TILE>(step * KEYS + r, w >> 2)) + (w & 3);
                    };
                    // the first such key of this lane's columns, a byte each
                    uint32_t bad = 0xffffffffu;
#pragma unroll 1
                    for (int r = r1 - 1; r >= r0; --r)
#pragma unroll 1
                        for (int w = lane; w < WORDS; w += 32) {
                            const uint32_t found = not_finite<FP8>(*word(r, w));
#pragma unroll
                            for (int i = 0; i < EACH; ++i)
                                if (found >> (i * BITS) & 1u) {
                                    const int at_bit = (w / 32 * EACH + i) * 8;
                                    bad = (bad & ~(0xffu << at_bit)) | (uint32_t)r << at_bit;
                                }
                        }
                    // The warps of all row groups look at the same keys, and clear
                    // the same words: none before all have looked, and none
                    // multiplies before all have cleared.  (These barriers do not
                    // hang on what the data is.)
                    if (C::kRg > 1)
                        named_barrier_sync(2 + kg, C::kRg * 32);
                    const bool any = __any_sync(0xffffffffu, bad != 0xffffffffu);
                    if (any) {
#pragma unroll 1
                        for (int r = r0; r < r1; ++r)
#pragma unroll 1
                            for (int w = lane; w < WORDS; w += 32) {
                                uint32_t *const x = word(r, w);
                                const uint32_t old = *x, found = not_finite<FP8>(old);
                                if (found)
                                    *x = old & ~(found * ((1u << BITS) - 1u));
                            }
                        fence_proxy_async_smem();  // before a tensor copy lands there
                    }
                    if (C::kRg > 1)
                        named_barrier_sync(2 + kg, C::kRg * 32);
                    else
                        __syncwarp();
                    if (any) {
#pragma unroll
                        for (int n = 0; n < DN; n += FP8 ? 2 : 1) {
                            const int w = FP8 ? n * 2 + t : n * 4 + t;
                            const uint32_t x = __shfl_sync(0xffffffffu, bad, w & 31) >> (FP8 ? 0 : w / 32 * 16);
#pragma unroll
                            for (int i = 0; i < EACH; ++i)
#pragma unroll
                                for (int hf = 0; hf < (RG == 0 ? 1 : 2); ++hf) {
                                    float &o = sums[FP8 ? n + i % 2 : n][hf * 2 + (FP8 ? i / 2 : i)];
                                    const int r = (int)(x >> (i * 8) & 0xffu);
                                    if (r != 0xff && kb + r < lim[hf])
                                        o = __int_as_float(0x7fffffff);
                                }
                        }
                    }
                }
                // values of 16 keys n*8 .. +15, columns c*8 .. +15
                auto load_v = [&](uint32_t (&f)[4], int c, int n) {
                    ldsm_x4_t(f, (v_u ^ (((c >> 1) & 3) << 5)) + (c >> 3) * BOXES + n * 8 * BOX);
                };
                if constexpr (FP8 || kByStep) {
#pragma unroll
                    for (int c = 0; c < DN; c += 2) {
                        float step_sums[2][ACC] = {};
                        float *const even = kByStep ? step_sums[0] : acc[kByStep ? 0 : c];
                        float *const odd = kByStep ? step_sums[1] : acc[kByStep ? 0 : c + 1];
                        if constexpr (FP8) {
                            // the transposed load pairs neighbouring elements of
                            // a key in each half: the low bytes of both halves
                            // make the even columns' operand, the high bytes the
                            // odd ones'
                            uint32_t f[4];
                            ldsm_x4_t(f, v_u ^ ((c >> 1) << 4));
#pragma unroll
                            for (int n = 0; n < 4; n += 2) {
                                const uint32_t x = __byte_perm(f[n], 0, 0x3120), y = __byte_perm(f[n + 1], 0, 0x3120);
                                add_pv(even, n, e4m3_to_f16(x), e4m3_to_f16(y));
                                add_pv(odd, n, e4m3_to_f16(x >> 16), e4m3_to_f16(y >> 16));
                            }
                        } else {
#pragma unroll
                            for (int n = 0; n < NT; n += 2) {
                                uint32_t f[4];
                                load_v(f, c, n);
                                add_pv(even, n, f[0], f[1]);
                                add_pv(odd, n, f[2], f[3]);
                            }
                        }
                        if constexpr (kByStep) {
                            add_to(sums[c], even, 1.f);
                            add_to(sums[c + 1], odd, 1.f);
                            if constexpr (FP8) {
                                add_to(sums[c], even + 4, kLow);
                                add_to(sums[c + 1], odd + 4, kLow);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; n += 2)
#pragma unroll
                        for (int c = 0; c < DN; c += 2) {
                            uint32_t f[4];
                            load_v(f, c, n);
                            add_pv(acc[c], n, f[0], f[1]);
                            add_pv(acc[c + 1], n, f[2], f[3]);
                        }
                }
            }
            if (--left == 0)
                break;
            release();
            ++at.j;
            if (!kByStep && ++fresh == kFlush)
                flush();
        }
        flush();

        // ---- the job's or the share's end: join the key groups' warps
        const bool last_tile = at.j == at.tiles - 1;
        const int next = next_pos<TILE>(at);
        const bool on = next < end;
        const bool whole = first_j == 0 && last_tile;
        // the next job's queries are asked for now, and arrive meanwhile
        const Place done = at;
        const int done_h = h_kv, done_row0 = row0, done_new = n_new;
        if (on) {
            advance<TILE>(a, at, next);
            load_q();
        }
        // through memory of their own where it fits, else through the stage,
        // once no warp reads the tile any more
        char *const rows = C::kOwnRows ? smem + C::kRowsAt : smem + stage * C::kStage;
        fence_proxy_async_smem();  // zeros in the stage, before a tensor copy lands there
        if (C::kOwnRows)
            release();
        named_barrier_sync(1, kWarps * 32);
        float *mine = reinterpret_cast<float *>(rows) + warp * C::kWarpRows * D;
#pragma unroll
        for (int hf = 0; hf < (RG == 0 ? 1 : 2); ++hf) {
            float l = l_run[hf];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int row = g + hf * 8;
            if (t == 0) {
                red_m[warp * C::kWarpRows + row] = m_run[hf] - kUp<FP8>;  // what the sums are relative to
                red_l[warp * C::kWarpRows + row] = l;
            }
#pragma unroll
            for (int n = 0; n < DN; n += FP8 ? 2 : 1) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = sums[n][hf * 2 + e];
                    if (FP8)
                        x[2 + e] = sums[n + 1][hf * 2 + e];
                }
                if (FP8) {
                    const int col = n * 8 + t * 4;
                    *reinterpret_cast<float4 *>(mine + row * D + (((col >> 3) ^ (row & 7)) << 3) + (col & 7)) =
                        make_float4(x[0], x[2], x[1], x[3]);
                } else {
                    *reinterpret_cast<float2 *>(mine + row * D + ((n ^ (row & 7)) << 3) + t * 2) = make_float2(x[0], x[1]);
                }
            }
        }
        if (!C::kOwnRows)
            fence_proxy_async_smem();
        named_barrier_sync(1, kWarps * 32);
        const int r = done_row0 + my_line;
        if (r < a.R) {
            const int row = my_line % C::kWarpRows, w0 = my_line / C::kWarpRows * C::kKg;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::kKg; ++w)
                top = fmaxf(top, red_m[(w0 + w) * C::kWarpRows + row]);
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f, o[CP];
#pragma unroll
            for (int e = 0; e < CP; ++e)
                o[e] = 0.f;
#pragma unroll
            for (int w = 0; w < C::kKg; ++w) {
                const float f = ex2_approx(red_m[(w0 + w) * C::kWarpRows + row] - ref);
                sum += f * red_l[(w0 + w) * C::kWarpRows + row];
                const float *src = reinterpret_cast<const float *>(rows) + ((w0 + w) * C::kWarpRows + row) * D;
#pragma unroll
                for (int e = 0; e < CP; e += 2) {
                    const int col = col0 + e * TPR;
                    const float2 x = *reinterpret_cast<const float2 *>(src + (((col >> 3) ^ (row & 7)) << 3) + (col & 7));
                    o[e] += f * x.x;
                    o[e + 1] += f * x.y;
                }
            }
            if (!whole) {
                const long long at_ws = (long long)(2 * blockIdx.x + (first_j == 0 ? 1 : 0)) * C::kRows + my_line;
#pragma unroll
                for (int e = 0; e < CP; e += 2)
                    *reinterpret_cast<float2 *>(a.ws_o + at_ws * D + col0 + e * TPR) = make_float2(o[e], o[e + 1]);
                if (col0 == 0)
                    a.ws_ml[at_ws] = make_float2(top, sum);
            } else if (a.Sq == 1 || r % a.Sq < done_new) {
                const float f = sum == 0.f ? 0.f : (FP8 ? a.cache.v_scale[done_h] : 1.f) / sum;
                const long long at_row = ((long long)done.b * a.Hkv + done_h) * a.R + r;
#pragma unroll
                for (int e = 0; e < CP; e += 2) {
                    if (a.out_bf16)
                        *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.out + at_row * D + col0 + e * TPR) =
                            pack_bf16(o[e] * f, o[e + 1] * f);
                    else
                        *reinterpret_cast<float2 *>((float *)a.out + at_row * D + col0 + e * TPR) =
                            make_float2(o[e] * f, o[e + 1] * f);
                }
                if (col0 == 0)
                    a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            }
        }
        if (first_j == 0 && !last_tile && tid == 0)  // the first part of a cut job: where is its last?
            a.ws_rec[blockIdx.x] = make_int4(done.b * a.Hkv * a.n_rt + done.hr, done_new, 0,
                                             shares.owner(done.pos + (done.tiles - 1 - done.j) * kUnits));
        if (!C::kOwnRows)
            release();
        if (!on)
            break;
    }
    named_barrier_arrive(kEndBarrier, kThreads);
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

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn get_encode_fn()
{
    static EncodeFn fn = []() -> EncodeFn {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? (EncodeFn)ptr : nullptr;
    }();
    return fn;
}

// The cache as [page][head][row][element], read in boxes of `rows` rows.
int encode_cache(CUtensorMap *m, const PagedView &c, void *base, int d, bool fp8, int rows, char *msg, size_t msg_len)
{
    const EncodeFn fn = get_encode_fn();
    if (!fn) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled is not available from the driver");
        return MERCURY_ECUDA;
    }
    const uint64_t es = fp8 ? 1 : 2, row = d * es;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {row, row * c.page_size, (cuuint64_t)c.page_stride * es};
    const cuuint32_t box[4] = {(cuuint32_t)((row < 128 ? row : 128) / es), (cuuint32_t)rows, 1, 1}, unit[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides,
                          box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(msg, msg_len, "cuTensorMapEncodeTiled (cache) failed (CUresult %d)", (int)r);
        return MERCURY_ECUDA;
    }
    return MERCURY_OK;
}

template <int D, bool FP8, int RG>
int launch(PagedArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    using C = Cfg<D, FP8, RG>;
    a.n_rt = (a.R + C::kRows - 1) / C::kRows;
    const long long keys = (long long)a.cache.max_pages * a.cache.page_size;
    const long long jobs = (long long)a.B * a.Hkv * a.n_rt;
    static_assert(kJobCost <= 2 * kUnits, "a job's cost counts as two tiles below");
    const long long most = ((keys + C::kTile - 1) / C::kTile + 2) * jobs;  // tiles, a job's cost included
    if (most > 0x7fffffffLL / kUnits) {
        snprintf(msg, msg_len, "too many key tiles for one call (%lld)", most);
        return MERCURY_EINVAL;
    }
    a.box_rows = 0;
    if (a.cache.page_size % 8 == 0) {
        for (a.box_rows = 8; a.box_rows < C::kTile && a.cache.page_size % (2 * a.box_rows) == 0;)
            a.box_rows *= 2;
        int rc = encode_cache(&a.map_k, a.cache, a.cache.k, D, FP8, a.box_rows, msg, msg_len);
        if (rc == MERCURY_OK)
            rc = encode_cache(&a.map_v, a.cache, a.cache.v, D, FP8, a.box_rows, msg, msg_len);
        if (rc != MERCURY_OK)
            return rc;
    }
    auto *kernel = attn_paged_kernel<D, FP8, RG>;
    KernelInfo ki;
    int rc = prepare_kernel((const void *)kernel, C::kSmem, &ki, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    if (ki.regs < kMinLaunchRegs) {
        // the register increase would wait for registers that do not exist
        snprintf(msg, msg_len, "paged attention kernel built with %d registers a thread, needs %d", ki.regs, kMinLaunchRegs);
        return MERCURY_ECUDA;
    }
    // What a call of this shape class with longer sequences needs is made now
    // too, so that it may be captured.
    auto *join = attn_paged_join_kernel<D, C::kRows>;
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
    const bool split = keys > C::kTile;
    void *ws = nullptr;
    if (split) {
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
    cudaError_t e = launch_chained(kernel, dim3(grid), kThreads, C::kSmem, stream, a);
    if (e == cudaSuccess && split) {
        // As many warps for a row as take its parts in one look, where the
        // jobs are alike; four at least, for jobs that are much longer than
        // the others.  (8 sequences of 16 rows, 64 jobs: 33.4 us, with all
        // eight warps 35.0, since twice the blocks take turns; with two 33.1,
        // but 73.7 instead of 73.0 in the 8-bit case above.)
        const long long parts = grid / jobs + 1;
        for (a.join_warps = 4; a.join_warps < kJoinWarps && a.join_warps * kJoinAhead < parts;)
            a.join_warps *= 2;
        const int rows = kJoinWarps / a.join_warps, used = C::kRows < a.R ? C::kRows : a.R;
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

template <int D, bool FP8>
int launch_rows(PagedArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    if (a.R <= 8)
        return launch<D, FP8, 0>(a, stream, msg, msg_len);
    if (a.R <= 16)
        return launch<D, FP8, 1>(a, stream, msg, msg_len);
    if (a.R <= 32)
        return launch<D, FP8, 2>(a, stream, msg, msg_len);
    return launch<D, FP8, 4>(a, stream, msg, msg_len);
}

}  // namespace

int launch_attn_paged(const void *q, const Strides &qs, const mercury_paged_cache &cache, const int *seq_lens,
                      const int *new_lens, int B, int Hq, int Sq, int causal, void *out, float *lse, int out_bf16,
                      unsigned long long wait_ns, int fault, cudaStream_t stream, char *msg, size_t msg_len)
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
    const bool fp8 = cache.elem == MERCURY_ELEM_E4M3;
    if (!fp8)
        a.cache.v_scale = nullptr;
    if (cache.d == 128)
        return fp8 ? launch_rows<128, true>(a, stream, msg, msg_len) : launch_rows<128, false>(a, stream, msg, msg_len);
    return fp8 ? launch_rows<64, true>(a, stream, msg, msg_len) : launch_rows<64, false>(a, stream, msg, msg_len);
}

int read_and_clear_paged_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    return read_and_clear_words(g_paged_err_word, g_paged_err_site, "paged attention", word, site, msg, msg_len);
}

}  // namespace mercury
