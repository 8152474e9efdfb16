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

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinThreads = 128;

struct PagedArgs {
    const __nv_bfloat16 *q;
    Strides qs;
    PagedView cache;
    const int *seq_lens, *new_lens;
    void *out;
    float *lse;
    float *ws_o;    // [2 * blocks][rows of a tile][d]
    float2 *ws_ml;  // [2 * blocks][rows of a tile]: maximum (log2 units), sum
    int4 *ws_rec;   // [blocks]: the split job whose first part the block holds, and its last block
    int B, Hq, Hkv, G, Sq, R, n_rt, causal, out_bf16;
    float scale_log2;
};

template <int D, bool FP8, int MT>
struct Cfg {
    static constexpr int kRowB = D * (FP8 ? 1 : 2);        // bytes of one key
    static constexpr int kKeys = kRowB == 256 ? 16 : 32;   // keys of a warp's tile
    static constexpr int kTile = kKeys * kWarps;           // keys of a block's tile
    static constexpr int kPart = kKeys * kRowB;            // bytes of a warp's K (or V) tile
    static constexpr int kStage = 2 * kPart;
    static constexpr int kStages = 196608 / (kWarps * kStage);
    static constexpr int kMt = MT == 0 ? 1 : MT;           // 16-row tiles
    static constexpr int kRows = MT == 0 ? 8 : 16 * MT;
    static constexpr int kPassRows = MT == 0 ? 8 : 16;     // rows reduced at a time
    static constexpr int kSmem = kWarps * kStages * kStage + kWarps * kRows * 8 + 64;
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
// that the eight rows of a matrix load hit eight different bank groups.
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

// A place in the list of all tiles of all jobs.
struct Place {
    int b, h, rt, j;       // sequence, KV head, row tile, tile of the job
    int tiles, keys, n;    // of sequence b: tiles of a job, keys, new tokens
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
    p.n = new_of(a, p.b);
    p.tiles = tiles_of<TILE>(p.keys, p.n);
}

// The next tile (the caller knows that there is one).
template <int TILE>
__device__ __forceinline__ void advance(const PagedArgs &a, Place &p)
{
    if (++p.j < p.tiles)
        return;
    p.j = 0;
    if (++p.rt < a.n_rt)
        return;
    p.rt = 0;
    if (++p.h < a.Hkv)
        return;
    p.h = 0;
    do {
        ++p.b;
        enter<TILE>(a, p);
    } while (p.tiles == 0);
}

// Number of tiles of sequences c*kThreads + [0, kThreads) and this thread's
// inclusive prefix of it.
template <int TILE>
__device__ __forceinline__ int scan_tiles(const PagedArgs &a, int c, int &incl, int *warp_sums)
{
    const int b = c * kThreads + threadIdx.x;
    int w = 0;
    if (b < a.B)
        w = tiles_of<TILE>(keys_of(a, b), new_of(a, b)) * a.Hkv * a.n_rt;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += x;
    }
    __syncthreads();
    if (lane == 31)
        warp_sums[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i == warp)
            incl += total;
        total += warp_sums[i];
    }
    return total;
}

template <int D, bool FP8, int MT>
__global__ void __launch_bounds__(kThreads, 1) attn_paged_kernel(const __grid_constant__ PagedArgs a)
{
    using C = Cfg<D, FP8, MT>;
    constexpr int ROWB = C::kRowB, KEYS = C::kKeys, TILE = C::kTile, NS = C::kStages, NT = KEYS / 8;
    constexpr int KK = D / 16, DN = D / 8;  // k-steps of Q.K, 8-column tiles of O
    extern __shared__ __align__(1024) char smem[];
    float *red_m = reinterpret_cast<float *>(smem + kWarps * NS * C::kStage);
    float *red_l = red_m + kWarps * C::kRows;
    int *sums = reinterpret_cast<int *>(red_l + kWarps * C::kRows);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this block's share of the tiles
    const int chunks = (a.B + kThreads - 1) / kThreads;
    int incl = 0, total = 0, first_total = 0;
    for (int c = 0; c < chunks; ++c) {
        int x;
        const int s = scan_tiles<TILE>(a, c, x, sums);
        if (c == 0) {
            incl = x;
            first_total = s;
        }
        total += s;
    }
    if (blockIdx.x == 0)
        for (int b = tid; b < a.B; b += kThreads) {
            if (__ldg(a.seq_lens + b) != keys_of(a, b))
                record_bounds(0x901);
            if (a.new_lens && __ldg(a.new_lens + b) != new_of(a, b))
                record_bounds(0x902);
        }
    // every working block gets a tile at least, so that the blocks that share a
    // job are neighbours
    const int blocks = min((int)gridDim.x, total);
    if ((int)blockIdx.x >= blocks) {
        if (tid == 0 && a.ws_rec)
            a.ws_rec[blockIdx.x] = make_int4(0, 0, 0, -1);
        return;
    }
    const int start = (int)((long long)blockIdx.x * total / blocks);
    const int end = (int)((long long)(blockIdx.x + 1) * total / blocks);
    {
        int base = 0;
        for (int c = 0; c < chunks; ++c) {
            int s = first_total;
            if (c > 0)
                s = scan_tiles<TILE>(a, c, incl, sums);
            if (start >= base && start < base + s) {
                const int b = c * kThreads + tid;
                const int w = b < a.B ? tiles_of<TILE>(keys_of(a, b), new_of(a, b)) * a.Hkv * a.n_rt : 0;
                const int off = start - (base + incl - w);
                __syncthreads();
                if (off >= 0 && off < w) {
                    sums[8] = b;
                    sums[9] = off;
                }
            }
            base += s;
        }
    }
    __syncthreads();
    Place at;
    at.b = sums[8];
    enter<TILE>(a, at);
    {
        const int off = sums[9], job = off / at.tiles;
        at.j = off - job * at.tiles;
        at.h = job / a.n_rt;
        at.rt = job - at.h * a.n_rt;
    }

    // ---- the ring of copied tiles: this warp's part of each block tile
    char *const ring = smem + warp * (NS * C::kStage);
    const uint32_t ring_u = smem_addr(ring);
    constexpr int CPR = ROWB / 16, RPP = 32 / CPR;  // chunks of a row, rows copied at a time
    const int my_row = lane / CPR, my_chunk = lane % CPR;
    Place ahead = at;
    int ahead_t = start;
    // the key row looked up by this lane for the next copy: page, row in it
    int look_page = -1, look_row = 0, look_h = 0;
    bool look_live = false;
    auto look_up = [&]() {
        look_live = ahead_t < end;
        if (!look_live)
            return;
        const int key = (ahead.j * kWarps + warp) * KEYS + lane % KEYS;
        look_page = -1;
        look_h = ahead.h;
        look_row = -1;
        if (key < ahead.keys) {
            const int pg = (int)((unsigned int)key / (unsigned int)a.cache.page_size);
            look_row = key - pg * a.cache.page_size;
            look_page = __ldg(a.cache.table + ahead.b * a.cache.table_stride + pg);
        }
        if (++ahead_t < end)
            advance<TILE>(a, ahead);
    };
    auto copy_tile = [&](int stage) {
        if (look_live) {
            long long off = -1;
            if (look_row >= 0) {
                if (look_page >= 0 && look_page < a.cache.num_pages)
                    off = (look_page * a.cache.page_stride +
                           ((long long)look_h * a.cache.page_size + look_row) * D) * (FP8 ? 1 : 2);
                else
                    record_bounds(0x903);
            }
            const uint32_t dst = ring_u + stage * C::kStage;
#pragma unroll
            for (int i = 0; i < KEYS / RPP; ++i) {
                const int r = i * RPP + my_row;
                const long long o = __shfl_sync(0xffffffffu, off, r);
                const long long src = max(o, 0LL) + my_chunk * 16;
                const uint32_t to = dst + chunk_at<ROWB>(r, my_chunk);
                copy16(to, a.cache.k + src, o >= 0);
                copy16(to + C::kPart, a.cache.v + src, o >= 0);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
        look_up();
        copy_tile(i);
    }
    look_up();

    // ---- the tiles
    uint32_t qf[C::kMt][KK][MT == 0 ? 2 : 4];
    float acc[C::kMt][DN][4];
    float m_run[C::kMt][2], l_run[C::kMt][2], s_mul[C::kMt][2];
    int lim[C::kMt][2];  // keys that each of this thread's rows sees
    int rec_last = -1;
    Place rec = at;
    bool fresh = true;
    int first_j = at.j;

    for (int i = start; i < end; ++i) {
        const int stage = (i - start) % NS;
        copy_wait<NS - 2>();
        __syncwarp();
        copy_tile((i - start + NS - 1) % NS);
        look_up();

        if (fresh) {
            fresh = false;
            first_j = at.j;
            float kmul = a.scale_log2;
            if (FP8)
                kmul *= __ldg(a.cache.k_scale + at.h);
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = at.rt * C::kRows + mt * 16 + g + hf * 8;
                    const bool live = r < a.R && (MT > 0 || hf == 0);
                    const int head = at.h * a.G + r / a.Sq, s = r % a.Sq;
                    m_run[mt][hf] = -INFINITY;
                    l_run[mt][hf] = 0.f;
                    lim[mt][hf] = a.causal ? at.keys - at.n + min(s, at.n - 1) + 1 : at.keys;
                    s_mul[mt][hf] = kmul;
                    if (MT == 0 && hf == 1)
                        continue;
                    const __nv_bfloat16 *src = a.q + at.b * a.qs.b + head * a.qs.h + s * a.qs.s;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        uint32_t x = 0, y = 0;
                        if (live) {
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
                        s_mul[mt][hf] = kmul * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                        for (int kk = 0; kk < KK; ++kk) {
                            uint32_t &x = qf[mt][kk][hf], &y = qf[mt][kk][MT == 0 ? 1 : 2 + hf];
                            x = pack_f16(bf16_lo(x) * f, bf16_hi(x) * f);
                            y = pack_f16(bf16_lo(y) * f, bf16_hi(y) * f);
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
            const uint32_t k_u = ring_u + stage * C::kStage, v_u = k_u + C::kPart;
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
                        uint32_t f[4];
                        const int r = n * 8 + (lane >> 4) * 8 + (lane & 7);
                        ldsm_x4(f, k_u + chunk_at<ROWB>(r, 2 * kk + ((lane >> 3) & 1)));
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
                    ldsm_x4(f, k_u + chunk_at<ROWB>(lane, kk));
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
            const int seen_by_all = a.causal ? at.keys - at.n + 1 : at.keys;
            const bool edge = kb + KEYS > seen_by_all;
            uint32_t p_hi[C::kMt][NT][2], p_lo[C::kMt][NT][2];
#pragma unroll
            for (int mt = 0; mt < C::kMt; ++mt) {
#pragma unroll
                for (int hf = 0; hf < (MT == 0 ? 1 : 2); ++hf) {
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &x = sc[mt][n][hf * 2 + e];
                            x *= s_mul[mt][hf];
                            if (edge && kb + n * 8 + t * 2 + e >= lim[mt][hf])
                                x = -INFINITY;
                            top = fmaxf(top, x);
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float m_old = m_run[mt][hf], m_new = fmaxf(m_old, top);
                    const float m_ref = m_new == -INFINITY ? 0.f : m_new;
                    if (__any_sync(0xffffffffu, m_new != m_old)) {
                        const float f = ex2(m_old - m_ref);
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
                    m_run[mt][hf] = m_new;
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float p0 = ex2(sc[mt][n][hf * 2] - m_ref), p1 = ex2(sc[mt][n][hf * 2 + 1] - m_ref);
                        sum += p0 + p1;
                        split2<FP8>(p0, p1, p_hi[mt][n][hf], p_lo[mt][n][hf]);
                    }
                    l_run[mt][hf] += sum;
                }
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
                            const int r = n * 8 + ((lane >> 3) & 1) * 8 + (lane & 7);
                            ldsm_x4_t(f, v_u + chunk_at<ROWB>(r, c + (lane >> 4)));
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
                        ldsm_x4_t(f, v_u + chunk_at<ROWB>(lane, c >> 1));
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
            if (edge && a.causal && at.n > 1) {
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
                for (int s = at.n - 1; s >= 0; --s) {
                    const int seen = at.keys - at.n + s + 1;
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
                            const int r = at.rt * C::kRows + mt * 16 + g;
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
        if (last_tile || i == end - 1) {
            const bool whole = first_j == 0 && last_tile;
            const int slot = 2 * blockIdx.x + (first_j == 0 ? 1 : 0);
            if (first_j == 0 && !last_tile) {
                // the block that holds the job's last tile
                const long long x = (long long)i + (at.tiles - 1 - at.j);
                rec = at;
                rec_last = (int)(((x + 1) * blocks - 1) / total);
            }
            constexpr int TPR = kThreads / C::kPassRows, CP = D / TPR;  // threads of a row, columns of a thread
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
                const int row = tid / TPR, col0 = (tid % TPR) * CP;
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
                    const float *src = reinterpret_cast<const float *>(smem + w * (NS * C::kStage) + stage * C::kStage) + row * D;
#pragma unroll
                    for (int e = 0; e < CP; e += 2) {
                        const int col = col0 + e;
                        const float2 x = *reinterpret_cast<const float2 *>(src + (((col >> 3) ^ (row & 7)) << 3) + (col & 7));
                        o[e] += f * x.x;
                        o[e + 1] += f * x.y;
                    }
                }
                const int r = at.rt * C::kRows + mt * 16 + row;
                if (!whole) {
                    const long long at_ws = (long long)slot * C::kRows + mt * 16 + row;
#pragma unroll
                    for (int e = 0; e < CP; e += 2)
                        *reinterpret_cast<float2 *>(a.ws_o + at_ws * D + col0 + e) = make_float2(o[e], o[e + 1]);
                    if (col0 == 0)
                        a.ws_ml[at_ws] = make_float2(top, sum);
                } else if (r < a.R && r % a.Sq < at.n) {
                    const float f = sum == 0.f ? 0.f : (FP8 ? __ldg(a.cache.v_scale + at.h) : 1.f) / sum;
                    const long long at_row = ((long long)at.b * a.Hq + at.h * a.G) * a.Sq + r;
#pragma unroll
                    for (int e = 0; e < CP; e += 2) {
                        if (a.out_bf16)
                            *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.out + at_row * D + col0 + e) =
                                pack_bf16(o[e] * f, o[e + 1] * f);
                        else
                            *reinterpret_cast<float2 *>((float *)a.out + at_row * D + col0 + e) =
                                make_float2(o[e] * f, o[e + 1] * f);
                    }
                    if (col0 == 0)
                        a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
                }
            }
            __syncthreads();
            fresh = true;
        }
        if (i + 1 < end)
            advance<TILE>(a, at);
    }
    copy_wait<0>();
    if (tid == 0 && a.ws_rec)
        a.ws_rec[blockIdx.x] = make_int4(rec.b, rec.h, rec.rt, rec_last);
}

// Joins the parts of a job that was cut between blocks: one thread block per
// (block that holds a first part, row of the tile).
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const __grid_constant__ PagedArgs a)
{
    constexpr int W = kJoinThreads / 32, PER = D / 32;
    __shared__ float part[W][D], red[W], sums[W];
    // every block waits, also those with nothing to do: the call is over only
    // when the first kernel is
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int first = blockIdx.x, row = blockIdx.y;
    const int4 rec = a.ws_rec[first];
    const int r = rec.z * ROWS + row;
    if (rec.w < 0 || r >= a.R || r % a.Sq >= new_of(a, rec.x))
        return;
    const int n = rec.w - first + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto slot_of = [&](int i) { return (long long)(2 * (first + i) + (i == 0 ? 1 : 0)) * ROWS + row; };
    float top = -INFINITY;
    for (int i = tid; i < n; i += kJoinThreads)
        top = fmaxf(top, a.ws_ml[slot_of(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w)
        top = fmaxf(top, red[w]);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e)
        o[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += W) {
        const long long s = slot_of(i);
        const float2 ml = a.ws_ml[s];
        const float f = ex2(ml.x - ref);
        sum += f * ml.y;
        const float *src = a.ws_o + s * D + lane * PER;
        float x[PER];
        if constexpr (PER == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(src);
            x[0] = v.x, x[1] = v.y;
        }
#pragma unroll
        for (int e = 0; e < PER; ++e)
            o[e] += f * x[e];
    }
#pragma unroll
    for (int e = 0; e < PER; ++e)
        part[warp][lane * PER + e] = o[e];
    if (lane == 0)
        sums[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w)
        sum += sums[w];
    const long long at_row = ((long long)rec.x * a.Hq + rec.y * a.G) * a.Sq + r;
    const float f = sum == 0.f ? 0.f : (a.cache.v_scale ? __ldg(a.cache.v_scale + rec.y) : 1.f) / sum;
    for (int c = tid; c < D; c += kJoinThreads) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            x += part[w][c];
        if (a.out_bf16)
            ((__nv_bfloat16 *)a.out)[at_row * D + c] = __float2bfloat16_rn(x * f);
        else
            ((float *)a.out)[at_row * D + c] = x * f;
    }
    if (tid == 0)
        a.lse[at_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D, bool FP8, int MT>
int launch(PagedArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    using C = Cfg<D, FP8, MT>;
    a.n_rt = (a.R + C::kRows - 1) / C::kRows;
    const long long keys = (long long)a.cache.max_pages * a.cache.page_size;
    const long long most = (keys + C::kTile - 1) / C::kTile * a.B * a.Hkv * a.n_rt;
    if (most > 0x7fffffffLL) {
        snprintf(msg, msg_len, "too many key tiles for one call (%lld)", most);
        return MERCURY_EINVAL;
    }
    auto *kernel = attn_paged_kernel<D, FP8, MT>;
    KernelInfo ki;
    int rc = prepare_kernel((const void *)kernel, C::kSmem, &ki, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    // one block per SM, and none that could not get a tile
    const unsigned grid = (unsigned)(most < ki.sms ? most : ki.sms);
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
    kernel<<<grid, kThreads, C::kSmem, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && split) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid, C::kRows);
        cfg.blockDim = dim3(kJoinThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<D, C::kRows>, a);
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
    return launch<D, FP8, 2>(a, stream, msg, msg_len);
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
    const bool fp8 = cache.elem == MERCURY_ELEM_E4M3;
    if (!fp8)
        a.cache.v_scale = nullptr;
    if (cache.d == 128)
        return fp8 ? launch_rows<128, true>(a, stream, msg, msg_len) : launch_rows<128, false>(a, stream, msg, msg_len);
    return fp8 ? launch_rows<64, true>(a, stream, msg, msg_len) : launch_rows<64, false>(a, stream, msg, msg_len);
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
