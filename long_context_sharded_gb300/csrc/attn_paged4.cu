// attn_paged4.cu -- attention of one new token (or a few) of every sequence
// over a paged cache held in 4 bits, split over the cache's length and joined.
//
// A cached key (or value) is a row of d/2 + d/16 bytes: d codes of e2m1, two a
// byte, and an e4m3 scale for each 16 of them; an element is code * scale *
// (the head's 32-bit scale).  code * scale has six bits and lies in fp16's
// range, so both products run on fp16 matrix instructions with exact operands,
// and all else is as with the other caches (attn_paged.cu): x_k = q.k /
// sqrt(d), LSE = ln sum exp x_k, O = sum exp(x_k - LSE) v_k, in one pass with
// a running maximum and sum, the keys of all sequences dealt to the blocks in
// equal shares of one line.
//
// What bounds it: 9/16 of a byte an element, 3.6 times less than 16-bit ones,
// leaves 200 cycles of an SM for 32 keys and values of 128, in which 128
// registers of them a lane are widened and scaled (64 lanes a cycle each) and
// multiplied.  So the layout spends instructions where there are fewest:
//   * keys and values are the instructions' first operands (16 rows), the
//     queries' rows their second (8): S' = K Q', O' = V' P'.  Up to 8 rows fill
//     an instruction (with the queries first half of it would idle), and more
//     rows share a tile's widened elements.
//   * the order of elements within a product's inner axis is free.  For S' a
//     thread takes two runs of a key's row, so that a byte widened is a
//     register of the operand as it stands, and two scales serve all of it;
//     for O' it takes one block of 16 elements of four pairs of keys, whose
//     codes are interleaved eight at a time before they are widened.
//   * S' leaves the instruction with a key a row, O' wants it with a key a
//     column: 8 x 8 transposes in registers.
//   * rows of 72 (36) bytes are copied as they lie, runs of a page at a time,
//     and keys are dealt to a warp's lanes such that rows read together start
//     in different banks.
//   * a warp takes 64 keys at a time where there are many, which leaves more to
//     overlap, and the job's queries lie in shared memory.
//
// Measured on a GB300, of the measured copy bandwidth (6680 GB/s): 16 sequences
// of 700 to 32K tokens, 32 query and 8 KV heads of 128: 62 us, 75 %; one of
// 128K, 64 query heads: 39 us, 58 %; with all products taken out these take 54
// and 31 us.  8 sequences of 20K to 32K, rows a KV head: 4 51 us, 72 %, 8 57 us,
// 16 88 us, 28 163 us, 56 311 us (above 16 each row tile widens for itself); heads
// of 64 (half the bytes): 35, 38, 58, 108 and 205 us.  The matrix instructions'
// unit is busy 26 to 32 % of the first two, and by the count of instructions
// those that widen and scale about as much each, in turn rather than together;
// two warps an SM quarter overlap them no further: 12 or 16 warps, longer windows
// of sums and other orders of the products were not faster.  One 4K sequence
// takes 8.2 us, of which bytes would be 0.7.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_split.cuh"
#include "ptx.cuh"

namespace mercury {

namespace {

// ROWS: rows of a row tile, 4, 8 or 16.  Every computing warp has all its rows
// and its own 32 H keys of each tile.  With four rows both terms of a weight
// share an instruction: columns 0 to 3 are the rows' first terms, 4 to 7 their
// second ones.
template <int D, int ROWS, int H>
struct Cfg {
    static constexpr int kWarps = 8;              // computing warps
    static constexpr int kThreads = (kWarps + kCopyWarps) * 32;
    static constexpr int kRowB = D / 2 + D / 16;  // bytes of one key
    static constexpr int kRun = D / 16;           // bytes of a run of a row that a thread takes
    static constexpr int kKeys = 32 * H;          // keys of a warp's step
    static constexpr int kTile = kKeys * kWarps;
    static constexpr int kPart = kTile * kRowB;
    static constexpr int kStage = 2 * kPart;
    static constexpr int kCols = ROWS == 16 ? 16 : 8;          // columns of S' and O'
    static constexpr int kRed = kWarps * ROWS * 8;             // each warp's maxima and sums
    static constexpr int kRowBytes = kWarps * kCols * D * 4;   // the warps' partial columns
    static constexpr bool kOwnRows = kRowBytes > kStage;       // in memory of their own, or in a stage
    static constexpr int kQueries = kCols * D * 2 + kCols * 4;  // the job's, as operands, and their factors
    static constexpr int kRoom = 232448 - 256 - kRed - kQueries - (kOwnRows ? kRowBytes : 0);
    static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
    static constexpr int kCtl = kStages * kStage + kRed + kStages * 16;
    static constexpr int kQueriesAt = (kCtl + 32 + 15) / 16 * 16;
    static constexpr int kPartsAt = kQueriesAt + kQueries;
    static constexpr int kSmem = kPartsAt + (kOwnRows ? kRowBytes : 0);
    static_assert(kStages >= 2 && kSmem <= 232448, "a stage to read and one on its way");
    static_assert(kTile % kUnits == 0, "whole eighths of a tile");
    // registers a thread after the split (setmaxnreg); their sum may not
    // exceed what the launch provides
    static constexpr uint32_t kRegsCopy = 72, kRegsCompute = 216;
    static constexpr int kMinLaunchRegs = (int)(kRegsCopy * 128 + kRegsCompute * kWarps * 32 + kThreads - 1) / kThreads;
};

// Untiled bulk copy global -> shared: both addresses and the size are
// multiples of 16 bytes; completion counted in bytes on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int I>
struct Byte {
    static constexpr int value = I;
};

// The transpose of an 8 x 8 matrix of 16-bit elements, two of a row a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// x in the bits of mask, y in the others.
__device__ __forceinline__ uint32_t select_bits(uint32_t x, uint32_t y, uint32_t mask)
{
    return (x & mask) | (y & ~mask);
}

// The key of a step that row g of the S' product's part c (0 to 3) stands for.
// Rows of 18 (9) words: these start in different banks for the lanes that a
// load takes together, both with a key for each g and with those of 2t, or 2t
// + 1, for each t.
template <int D>
__device__ __forceinline__ int key_at(int g)
{
    return 4 * (D == 128 ? g ^ (g >> 2) : g);
}

// The copying warps: every tile of the share into the ring, a stage as soon as
// the computing warps have left it.  A tile's runs of box_rows keys, each in
// one page, are dealt to the lanes of the four warps in turn.
template <int D, int ROWS, int H>
__device__ __forceinline__ void copy_tiles(const PagedArgs &a, Place at, int end, char *smem, uint64_t *full,
                                           uint64_t *empty, Stop *stop, int warp, int lane)
{
    using C = Cfg<D, ROWS, H>;
    constexpr int ROWB = C::kRowB, TILE = C::kTile, NS = C::kStages;
    const int first = (lane * kCopyWarps + warp) * a.box_rows;  // this lane's run
    // its page, asked for a tile ahead
    int entry = -1;
    auto key_of = [&]() { return at.j * TILE + first; };
    auto look_up = [&]() {
        if (first < TILE && key_of() < at.keys)
            entry = a.cache.table[at.b * a.cache.table_stride + page_of(a.cache, key_of())];
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
        const int key = key_of(), row = key - page_of(a.cache, key) * a.cache.page_size;
        const bool live = first < TILE && key < at.keys;
        const bool good = live && entry >= 0 && entry < a.cache.num_pages;
        wait_phase(empty + stage, phase, a.wait_ns, stop);
        if (__any_sync(0xffffffffu, stopped(stop)))
            break;
        if (live && !good) {  // such keys count as zeros
            record_bounds(0x903);
            for (int i = 0; i < a.box_rows * ROWB; i += 16) {
                const uint32_t to = smem_u32(part) + first * ROWB + i;
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
            const long long from = entry * a.cache.page_stride + ((long long)h * a.cache.page_size + row) * ROWB;
            const uint32_t to = smem_u32(part) + first * ROWB, bytes = a.box_rows * ROWB;
            bulk_load(to, a.cache.k + from, bytes, smem_u32(full + stage));
            bulk_load(to + C::kPart, a.cache.v + from, bytes, smem_u32(full + stage));
        }
        ++sent;
        if (!on)
            break;
        advance<TILE>(a, at, next);
        look_up();
        if (at.j == 0 && warp == 0) {
            // a new job: its queries into L2 by the time the computing warps
            // get there
            const int h1 = a.n_rt == 1 ? at.hr : at.hr / a.n_rt, row0 = (at.hr - h1 * a.n_rt) * ROWS;
            for (int r = row0 + lane; r < min(row0 + ROWS, a.R); r += 32) {
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
    named_barrier_sync(kEndBarrier, C::kThreads);
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
        if (lane == 0)
            mbar_arrive(full + i % NS);
    for (int i = max(most - NS, 0); i < most; ++i) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(full + i % NS, i / NS & 1) && globaltimer_ns() - t0 <= a.wait_ns)
            ;
    }
}

// A run of kRun bytes (8 or 4) from shared memory.
template <int N>
__device__ __forceinline__ void load_run(uint32_t (&w)[N], const char *p)
{
    if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// Where element col of a partial row lies: its 16-byte chunks permuted by the
// row, so that the rows that a store takes together hit different banks.
__device__ __forceinline__ int part_at(int row, int col)
{
    return (((col >> 2) ^ (((row >> 1) & 3) | (row & 1) << 2)) << 2) + (col & 3);
}

template <int D, int ROWS, int H>
__global__ void __launch_bounds__(Cfg<D, ROWS, H>::kThreads, 1) attn_paged4_kernel(const __grid_constant__ PagedArgs a)
{
    using C = Cfg<D, ROWS, H>;
    constexpr int ROWB = C::kRowB, KEYS = C::kKeys, TILE = C::kTile, NS = C::kStages, kWarps = C::kWarps;
    constexpr int RUN = C::kRun, RW = RUN / 4;  // bytes and words of a thread's run of a row
    constexpr int KK = D / 16, DT = D / 16;     // k-steps of S', 16-row tiles of O'
    constexpr bool TWO = ROWS == 4;             // two terms in one instruction
    constexpr int NR = C::kCols / 8, TERMS = TWO ? 1 : 2;
    extern __shared__ __align__(1024) char smem[];
    float *const red_m = reinterpret_cast<float *>(smem + NS * C::kStage);
    float *const red_l = red_m + kWarps * ROWS;
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + NS * C::kStage + C::kRed);
    uint64_t *const empty = full + NS;
    Stop *const stop = reinterpret_cast<Stop *>(smem + C::kCtl);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        stop->now = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, kCopyWarps);
            mbar_init(empty + i, kWarps);
        }
        fence_mbar_init();
    }
    // The parameters that the share is found with: fetched while the kernel
    // before this one still runs, where their latency costs nothing.
    asm volatile("" ::"l"(a.seq_lens), "l"(a.new_lens), "r"(a.B), "r"(a.Hkv), "r"(a.n_rt), "r"(a.cache.max_pages),
                 "r"(a.cache.page_size), "l"(a.cache.table), "l"(a.q), "r"(a.Sq), "l"(a.ws_rec), "l"(a.wait_ns));
    chain_wait();
    __syncthreads();
    if (tid == 0 && a.ws_rec)
        a.ws_rec[blockIdx.x] = make_int4(0, 0, 0, -1);
    if (blockIdx.x == 0)
        for (int b = tid; b < a.B; b += C::kThreads) {
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
        regs_dec<C::kRegsCopy>();
        copy_tiles<D, ROWS, H>(a, at, end, smem, full, empty, stop, warp - kWarps, lane);
        return;
    }

    // ---- the computing warps
    regs_inc<C::kRegsCompute>();
    const int g = lane >> 2, t = lane & 3;
    // Row g of the second operand is query row nr * 8 + g (of four rows each is
    // there twice); of S' and O' this thread has the columns nr * 8 + 2t and + 1.
    // The operands and the rows' factors lie in shared memory (kept in registers
    // by every warp, they left room for no more than 12 of them): warp nr loads
    // those of its rows when a job is known, and puts them there between the two
    // barriers of the job before.
    uint2 *const queries = reinterpret_cast<uint2 *>(smem + C::kQueriesAt);  // [nr][k-step][lane]
    float *const factors = reinterpret_cast<float *>(queries + NR * KK * 32);  // [column]
    int h_kv, row0, n_new;  // of the current job: KV head, first row, new tokens
    uint2 q[KK];
    float k_scale = 1.f;
    auto load_q = [&]() {
        h_kv = a.n_rt == 1 ? at.hr : at.hr / a.n_rt;
        row0 = (at.hr - h_kv * a.n_rt) * ROWS;
        n_new = new_of(a, at.b);
        if (warp < NR) {
            k_scale = a.cache.k_scale[h_kv];
            const int r = row0 + (TWO ? g & 3 : warp * 8 + g);
            const int head = a.Sq == 1 ? r : r / a.Sq, s = r - head * a.Sq;
            const __nv_bfloat16 *src = a.q + at.b * a.qs.b + (h_kv * a.G + head) * a.qs.h + s * a.qs.s;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                q[kk] = r < a.R ? *reinterpret_cast<const uint2 *>(src + kk / (KK / 2) * (D / 2) + t * (D / 8) + kk % (KK / 2) * 4)
                                : make_uint2(0, 0);
        }
    };
    auto put_q = [&]() {
        if (warp >= NR)
            return;
        // a factor of at least 2^-120, so that a masked score stays -inf
        // under it; the scale's sign goes to the queries
        float kmul = a.scale_log2 * k_scale;
        const uint32_t flip = kmul < 0.f ? 0x80008000u : 0u;
        kmul = fabsf(kmul);
        // The queries are taken to fp16: scaled by a power of two that
        // brings the row's largest element to [2^14, 2^15), their 8 bits
        // fit exactly down to 2^-28 of it.
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(q[kk].x)), fabsf(bf16_hi(q[kk].x))),
                                   fmaxf(fabsf(bf16_lo(q[kk].y)), fabsf(bf16_hi(q[kk].y)))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent of 2^(14 - e), kept where both it and its inverse are normal
        int up = 14 + 127 - (int)(__float_as_uint(top) >> 23);
        up = min(max(up, -110), 110);
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
        const float mul = kmul * __uint_as_float((uint32_t)(127 - up) << 23);
        if (t == 0)
            factors[warp * 8 + g] = mul < 7.5e-37f ? 7.5e-37f : mul;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            queries[(warp * KK + kk) * 32 + lane] = make_uint2(pack_f16(bf16_lo(q[kk].x) * f, bf16_hi(q[kk].x) * f) ^ flip,
                                                               pack_f16(bf16_lo(q[kk].y) * f, bf16_hi(q[kk].y) * f) ^ flip);
    };
    load_q();
    put_q();
    named_barrier_sync(1, kWarps * 32);

    // O' of 16 elements a thread, by tiles: [0, 1] of the even ones, [2, 3] of
    // the odd.  The matrix unit truncates, so its own sums are short, 32 keys',
    // and are added to these by rounding additions.
    float sums[NR][DT][4];
    float m_run[NR][2], l_run[NR][2], l_rest[NR][2], s_mul[NR][2];  // l_rest: what l_run's roundings left out
    int lim[NR][2];                                                // keys that each column sees
    const int key_g = key_at<D>(g), key_x = key_at<D>(2 * t), key_y = key_at<D>(2 * t + 1);
    const char *const k_lane = smem + (warp * KEYS + key_g) * ROWB;
    const char *const v_lane = smem + C::kPart + warp * KEYS * ROWB;
    // which bytes of a row's scales this thread's runs have, and of two rows' its block
    const uint32_t k_pick = D == 128 ? t | (4 + t) << 4 : t / 2 | (2 + t / 2) << 4;
    const uint32_t v_pick = D == 128 ? (g & 3) | (4 + (g & 3)) << 4 | 0x4400 : g / 2 | (4 + g / 2) << 4 | 0x4400;
    const float whole_p = t < 2 ? 1.f : 1 << kLowShift, less_p = t < 2 ? 0.f : 1 << kLowShift;
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
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s_mul[nr][e] = factors[nr * 8 + 2 * t + e];
                m_run[nr][e] = -INFINITY;
                l_run[nr][e] = 0.f;
                l_rest[nr][e] = 0.f;
                const int s = (row0 + (TWO ? (2 * t + e) & 3 : nr * 8 + 2 * t + e)) % a.Sq;
                lim[nr][e] = a.causal ? at.keys - n_new + min(s, n_new - 1) + 1 : at.keys;
            }
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sums[nr][i][e] = 0.f;
        }

        for (;;) {
            wait_phase(full + stage, phase, a.wait_ns, stop);
            const int kb = at.j * TILE + warp * KEYS;
            if (kb < at.keys) {
                const char *const k_s = k_lane + stage * C::kStage, *const v_s = v_lane + stage * C::kStage;
                // ---- S' = K Q'
                float sc[H][NR][2][4];
#pragma unroll
                for (int h0 = 0; h0 < H; ++h0) {
                    constexpr int HN = 1;
                    // Part j: 16 keys, rows g and g + 8 of the product, keys key_g + 2m and
                    // + 1.  The parts' products are independent of one another, and go
                    // in turn.
                    uint32_t x[2 * HN][2][2][RW], s[2 * HN][2][2];  // [part][row][run]
#pragma unroll
                    for (int j = 0; j < 2 * HN; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const char *const row = k_s + (32 * (h0 + j / 2) + 2 * (j & 1) + i) * ROWB;
                            load_run(x[j][i][0], row + t * RUN);
                            load_run(x[j][i][1], row + D / 4 + t * RUN);
                            uint32_t all[RW];  // the row's scales
                            load_run(all, row + D / 2);
                            const uint32_t both = e4m3_to_f16(__byte_perm(all[0], all[RW - 1], k_pick));
                            s[j][i][0] = __byte_perm(both, 0, 0x1010);
                            s[j][i][1] = __byte_perm(both, 0, 0x3232);
                        }
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int w = 0; w < RW; ++w) {
                            const int kk = r * (KK / 2) + w * 2;
                            uint2 q[NR][2];
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    q[nr][i] = queries[(nr * KK + kk + i) * 32 + lane];
#pragma unroll
                            for (int j = 0; j < 2 * HN; ++j) {
                                const uint32_t x0 = x[j][0][r][w], x1 = x[j][1][r][w];
                                uint32_t f[8] = {e2m1_to_f16<0>(x0), e2m1_to_f16<0>(x1), e2m1_to_f16<1>(x0), e2m1_to_f16<1>(x1),
                                                 e2m1_to_f16<2>(x0), e2m1_to_f16<2>(x1), e2m1_to_f16<3>(x0), e2m1_to_f16<3>(x1)};
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    f[i] = mul_f16(f[i], s[j][i & 1][r]);
#pragma unroll
                                for (int nr = 0; nr < NR; ++nr) {
                                    float *const d = sc[h0 + j / 2][nr][j & 1];
                                    if (kk == 0)
                                        mma_first<true>(d, f[0], f[1], f[2], f[3], q[nr][0].x, q[nr][0].y);
                                    else
                                        mma<true>(d, f[0], f[1], f[2], f[3], q[nr][0].x, q[nr][0].y);
                                    mma<true>(d, f[4], f[5], f[6], f[7], q[nr][1].x, q[nr][1].y);
                                }
                            }
                        }
                }
                // Of part c of 32 keys, for O', the thread has block g of keys key_x + c
                // and key_y + c, the inner axis's columns 2t and 2t + 1: their scales.
                uint32_t vs[H][4];
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const char *const row = v_s + (32 * h + c) * ROWB + D / 2 + (D == 128 ? g / 4 * 4 : 0);
                        vs[h][c] = __byte_perm(*reinterpret_cast<const uint32_t *>(row + key_x * ROWB),
                                               *reinterpret_cast<const uint32_t *>(row + key_y * ROWB), v_pick);
                    }
                const int seen_by_all = a.causal ? at.keys - n_new + 1 : at.keys;
                if (kb + KEYS > seen_by_all) {
                    // The masked keys of a column count as -inf.  Scales of values
                    // behind the last key may be anything: those count as zeros.  So
                    // do those of NaN that only some rows see, whose product with a
                    // weight of 0 would be NaN; the rows that see one get NaN in its
                    // block's elements.
                    int bad = 0x7fffffff;
#pragma unroll
                    for (int h = 0; h < H; ++h) {
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (kb + 32 * h + key_g + 2 * m + (e >> 1) >= lim[nr][e & 1])
                                        sc[h][nr][m][e] = -INFINITY;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int key = kb + 32 * h + (i ? key_y : key_x) + c;
                                const bool nan = (vs[h][c] >> (8 * i) & 0x7fu) == 0x7fu;
                                if (key >= at.keys || (nan && a.causal && n_new > 1)) {
                                    vs[h][c] &= i ? 0x00ffu : 0xff00u;
                                    if (key < at.keys)
                                        bad = min(bad, key);
                                }
                            }
                    }
                    bad = min(bad, __shfl_xor_sync(0xffffffffu, bad, 1));
                    bad = min(bad, __shfl_xor_sync(0xffffffffu, bad, 2));
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (bad < lim[nr][e]) {
#pragma unroll
                                for (int i = 0; i < DT; ++i)
                                    sums[nr][i][e] = sums[nr][i][2 + e] = __int_as_float(0x7fffffff);
                            }
                }
                // The maximum moves only when a score exceeds it by 2^kGrow: sum and O
                // share whatever reference the terms were taken with, and the
                // reduction and the rescaling stay off the common path.
                bool grow = false;
                float top[NR][2];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = -INFINITY;
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            x = fmaxf(x, fmaxf(fmaxf(sc[h][nr][0][e], sc[h][nr][0][2 + e]), fmaxf(sc[h][nr][1][e], sc[h][nr][1][2 + e])));
                        top[nr][e] = x * s_mul[nr][e];
                        grow |= top[nr][e] > m_run[nr][e] + kGrow<true>;
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = top[nr][e];
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            x = fmaxf(x, m_run[nr][e]);
                            const float f = x == -INFINITY ? 1.f : ex2_approx(m_run[nr][e] - x);
                            m_run[nr][e] = x;
                            l_run[nr][e] *= f;
                            l_rest[nr][e] *= f;
#pragma unroll
                            for (int i = 0; i < DT; ++i) {
                                sums[nr][i][e] *= f;
                                sums[nr][i][2 + e] *= f;
                            }
                        }
                }
                // ---- P' as two fp16 terms, a key a column: p[..][m][half][term]
                uint32_t p[H][NR][2][2][TERMS];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float ref[2], sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        ref[e] = m_run[nr][e] == -INFINITY ? 0.f : kUp<true> - m_run[nr][e];
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float p0 = ex2_approx(fmaf(sc[h][nr][m][2 * i], s_mul[nr][0], ref[0]));
                                const float p1 = ex2_approx(fmaf(sc[h][nr][m][2 * i + 1], s_mul[nr][1], ref[1]));
                                sum[0] += p0;
                                sum[1] += p1;
                                uint32_t (&to)[TERMS] = p[h][nr][m][i];
                                if constexpr (TWO) {
                                    // p, or in the upper columns what its first term leaves, 2^kLowShift times as large
                                    const uint32_t w = pack_f16(p0, p1);
                                    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                                    to[0] = transpose8(pack_f16(fmaf(p0, whole_p, -x.x * less_p), fmaf(p1, whole_p, -x.y * less_p)));
                                } else {
                                    uint32_t term[2];
                                    split<true>(p0, p1, term);
                                    to[0] = transpose8(term[0]);
                                    to[TERMS - 1] = transpose8(term[1]);
                                }
                            }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // with what is left of earlier roundings: equal weights,
                        // small beside the sum, all round the same way
                        const float x = sum[e] + l_rest[nr][e];
                        const float l = l_run[nr][e] + x;
                        l_rest[nr][e] = x - (l - l_run[nr][e]);
                        l_run[nr][e] = l;
                    }
                }
                // ---- O' += V' P'
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    uint32_t scale[4], lo[4][RW], hi[4][RW];  // codes of both keys side by side: even elements, odd ones
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        scale[c] = e4m3_to_f16(vs[h][c]);
                        uint32_t x[RW], y[RW];
                        load_run(x, v_s + (32 * h + key_x + c) * ROWB + g * RUN);
                        load_run(y, v_s + (32 * h + key_y + c) * ROWB + g * RUN);
#pragma unroll
                        for (int w = 0; w < RW; ++w) {
                            lo[c][w] = select_bits(x[w], y[w] << 4, 0x0f0f0f0fu);
                            hi[c][w] = select_bits(x[w] >> 4, y[w], 0x0f0f0f0fu);
                        }
                    }
                    auto tile_of = [&](int i, int w, auto byte) {
                        constexpr int I = decltype(byte)::value;
                        float d[NR][TERMS][4];
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t a0 = mul_f16(e2m1_to_f16<I>(lo[2 * m][w]), scale[2 * m]);
                            const uint32_t a1 = mul_f16(e2m1_to_f16<I>(hi[2 * m][w]), scale[2 * m]);
                            const uint32_t a2 = mul_f16(e2m1_to_f16<I>(lo[2 * m + 1][w]), scale[2 * m + 1]);
                            const uint32_t a3 = mul_f16(e2m1_to_f16<I>(hi[2 * m + 1][w]), scale[2 * m + 1]);
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int term = 0; term < TERMS; ++term) {
                                    const uint32_t b0 = p[h][nr][m][0][term], b1 = p[h][nr][m][1][term];
                                    if (m == 0)
                                        mma_first<true>(d[nr][term], a0, a1, a2, a3, b0, b1);
                                    else
                                        mma<true>(d[nr][term], a0, a1, a2, a3, b0, b1);
                                }
                        }
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            add_to(sums[nr][i], d[nr][0], 1.f);
                            if constexpr (!TWO)
                                add_to(sums[nr][i], d[nr][TERMS - 1], kLow);
                        }
                    };
#pragma unroll
                    for (int w = 0; w < RW; ++w) {
                        tile_of(w * 4, w, Byte<0>());
                        tile_of(w * 4 + 1, w, Byte<1>());
                        tile_of(w * 4 + 2, w, Byte<2>());
                        tile_of(w * 4 + 3, w, Byte<3>());
                    }
                }
            }
            if (--left == 0)
                break;
            release();
            ++at.j;
        }

        // ---- the job's or the share's end: join the warps
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
        // through memory of their own, or through the stage, once no warp reads
        // the tile any more
        float *const rows = reinterpret_cast<float *>(C::kOwnRows ? smem + C::kPartsAt : smem + stage * C::kStage);
        if (C::kOwnRows)
            release();
        named_barrier_sync(1, kWarps * 32);
        if (on)
            put_q();  // no warp reads the last job's any more
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nr][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int row = nr * 8 + 2 * t + e;
                if (g == 0 && row < ROWS) {
                    red_m[warp * ROWS + row] = m_run[nr][e] - kUp<true>;  // what the sums are relative to
                    red_l[warp * ROWS + row] = l;
                }
                float *const mine = rows + (warp * C::kCols + row) * D;
#pragma unroll
                for (int i = 0; i < DT; i += 2)
                    *reinterpret_cast<float4 *>(mine + part_at(row, g * 2 * RUN + 2 * i)) =
                        make_float4(sums[nr][i][e], sums[nr][i][2 + e], sums[nr][i + 1][e], sums[nr][i + 1][2 + e]);
            }
        if (!C::kOwnRows)
            fence_proxy_async_smem();
        named_barrier_sync(1, kWarps * 32);
        for (int u = tid; u < ROWS * (D / 2); u += kWarps * 32) {
            const int row = u / (D / 2), col = u % (D / 2) * 2, r = done_row0 + row;
            if (r >= a.R)
                continue;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top = fmaxf(top, red_m[w * ROWS + row]);
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2_approx(red_m[w * ROWS + row] - ref);
                sum += f * red_l[w * ROWS + row];
                float2 x = *reinterpret_cast<const float2 *>(rows + (w * C::kCols + row) * D + part_at(row, col));
                if constexpr (TWO) {
                    const float2 y = *reinterpret_cast<const float2 *>(rows + (w * C::kCols + row + 4) * D + part_at(row + 4, col));
                    x = make_float2(x.x + kLow * y.x, x.y + kLow * y.y);
                }
                o0 += f * x.x;
                o1 += f * x.y;
            }
            if (!whole) {
                const long long at_ws = (long long)(2 * blockIdx.x + (first_j == 0 ? 1 : 0)) * ROWS + row;
                *reinterpret_cast<float2 *>(a.ws_o + at_ws * D + col) = make_float2(o0, o1);
                if (col == 0)
                    a.ws_ml[at_ws] = make_float2(top, sum);
            } else if (a.Sq == 1 || r % a.Sq < done_new) {
                const float f = sum == 0.f ? 0.f : a.cache.v_scale[done_h] / sum;
                const long long at_row = ((long long)done.b * a.Hkv + done_h) * a.R + r;
                if (a.out_bf16)
                    *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.out + at_row * D + col) = pack_bf16(o0 * f, o1 * f);
                else
                    *reinterpret_cast<float2 *>((float *)a.out + at_row * D + col) = make_float2(o0 * f, o1 * f);
                if (col == 0)
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
    named_barrier_arrive(kEndBarrier, C::kThreads);
}

template <int D, int ROWS, int H>
int launch(PagedArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    using C = Cfg<D, ROWS, H>;
    if constexpr (ROWS <= 8) {
        // A call of other lengths may take the other step: its kernel is made
        // ready now too, so that such a call may be captured.
        KernelInfo other;
        const int rc = prepare_kernel((const void *)attn_paged4_kernel<D, ROWS, 3 - H>, Cfg<D, ROWS, 3 - H>::kSmem, &other, msg,
                                      msg_len);
        if (rc != MERCURY_OK)
            return rc;
    }
    long long most;
    const int rc = count_tiles<ROWS, C::kTile>(a, &most, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    // runs of a power of two of keys that divides page_size (a multiple of 8) and the tile
    for (a.box_rows = 8; C::kTile % (2 * a.box_rows) == 0 && a.cache.page_size % (2 * a.box_rows) == 0;)
        a.box_rows *= 2;
    return launch_split<D, ROWS, C::kTile>(a, most, attn_paged4_kernel<D, ROWS, H>, C::kSmem, C::kThreads, C::kMinLaunchRegs,
                                               stream, msg, msg_len);
}

template <int D>
int launch_rows(PagedArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    if (a.R > 8)
        return launch<D, 16, 1>(a, stream, msg, msg_len);
    // Steps of 64 keys leave more to overlap than of 32, but tiles of 512 keys
    // go round the SMs only where there are many (one sequence of 128K: 38.6 us
    // instead of 41.1; of 4K, 64 tiles of 512: 9.2 instead of 8.2).
    int sms = 0;
    const int rc = device_sm_count(&sms);
    if (rc != MERCURY_OK)
        return rc;
    const long long tiles = (long long)a.cache.max_pages * a.cache.page_size / 512 * a.B * a.Hkv;
    if (tiles < 2 * sms)
        return a.R <= 4 ? launch<D, 4, 1>(a, stream, msg, msg_len) : launch<D, 8, 1>(a, stream, msg, msg_len);
    return a.R <= 4 ? launch<D, 4, 2>(a, stream, msg, msg_len) : launch<D, 8, 2>(a, stream, msg, msg_len);
}

}  // namespace

int launch_attn_paged4(const void *q, const Strides &qs, const mercury_paged_cache &cache, const int *seq_lens,
                       const int *new_lens, int B, int Hq, int Sq, int causal, void *out, float *lse, int out_bf16,
                       unsigned long long wait_ns, int fault, cudaStream_t stream, char *msg, size_t msg_len)
{
    PagedArgs a = paged_args(q, qs, cache, seq_lens, new_lens, B, Hq, Sq, causal, out, lse, out_bf16, wait_ns, fault);
    return cache.d == 128 ? launch_rows<128>(a, stream, msg, msg_len) : launch_rows<64>(a, stream, msg, msg_len);
}

int read_and_clear_paged4_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    return read_and_clear_words(g_paged_err_word, g_paged_err_site, "4-bit paged attention", word, site, msg, msg_len);
}

}  // namespace mercury
