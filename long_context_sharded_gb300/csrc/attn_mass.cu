// attn_mass.cu -- the attention weight that every cached key got from the
// newest tokens of its sequence.
//
// out[b][h][k] = mass[b][h][k] + sum over the rows r of KV head h (its query
// heads' new tokens) of exp(q_r.k / sqrt(d) - lse_r), over the rows that see
// key k; lse_r is what attention gave.
//
// Each key is read once, values not at all.  A key belongs to one warp (or, of
// many rows, to two, which add up half of them each), in a fixed order: no
// atomics, the same bits in every run.  All tiles of all heads, in order, are
// dealt to the blocks in equal contiguous shares, counted on the device from
// seq_lens.
//
// Few rows (a decode step, a few drafted tokens): warp-level products.  Keys
// are the first operand (16 rows), straight from memory into registers: the
// order of elements within a product's inner axis is free, so a lane takes
// whole 16-byte (8- or 4-byte) runs of two keys, and the queries, held in shared
// memory as operands, in the same order.  All rows of the head go over the
// registers that hold 16 keys, so further rows cost no further reads, and an 8-
// or 4-bit key is widened once.  More than 48 or 64 rows: the tensor unit, below.
//
// Measured on a GB300, of the measured copy bandwidth (6680 GB/s) or the
// product's rate: one token of 8 sequences of 20K to 32K, 32 query and 8 KV
// heads of 128: 16-bit keys 69 us, 95 %; e4m3 50 us, 67 %, e2m1 51 us, 37 %:
// not by bytes, but since each warp looks up, loads and widens its own next tile,
// one ahead (attention over 4 bits, whose copying warps fill a ring, reads twice the
// bytes in that time; 16-bit keys take 320 instructions for 16 keys of a warp).  Rows a KV head, 16
// bits: 16 73 us, 32 86, 64 122, 128 157, 256 221 (501 TFLOP/s); e2m1 57, 74,
// 86, 106, 153; e4m3 55, 72, 105, 106, 157; heads of 64, one token: 41, 36 and 40 us.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_split.cuh"
#include "ptx.cuh"

namespace mercury {

namespace {

constexpr int kMassWarps = 8;
constexpr int kMassThreads = kMassWarps * 32;
constexpr int kMassTile = kMassWarps * 16;  // keys of a block's tile
constexpr int kMassRows = 64;               // most rows that go by warps; more by the tensor unit,
constexpr int kWideRows = 256;              // so many a launch

struct MassArgs {
    PagedArgs p;        // q, qs, cache, seq_lens, new_lens, B, Hkv, G, Sq, R, causal
    const float *lse;   // [B][Hkv][R]
    const float *mass;  // [B][Hkv][width], or none
    float *out;         // the same
    long long width;
    int r0, rows;       // this launch's rows of each head
    int wide;           // rows of the tensor unit's product, or 0
    float mul, mul_lo;  // log2(e) / sqrt(d), and what its rounding leaves out
    int head0, step0;   // r0's head and new token
    int per_sq;         // 2^16 / Sq, rounded up
};

// A row of queries: a weight is 2^(score * mul + nl) * rest.  nl, lse in log2
// units, would cost the weight its rounding (lse 20: 1e-6), and mul's rounding
// as much; so nl is taken with the rounded mul, which leaves of the latter what
// score and lse differ by, and what nl's rounding leaves out goes to rest.
// A row that counts nothing: nl = -inf, rest = 0.
struct Row {
    float mul, nl, rest;
    int step;  // of the new tokens
};

// 16 keys as the first operand: rows g and g + 8.
template <int ELEM, int D>
struct Keys;

template <int D>
struct Keys<MERCURY_ELEM_BF16, D> {
    static constexpr int kRun = 8;  // elements of a lane's run
    static constexpr bool kF16 = false;
    static constexpr int kRowB = 2 * D;
    uint4 w[2][D / 32];
    __device__ __forceinline__ void load(int i, const char *row, int t)
    {
        if (!row) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                w[i][j] = make_uint4(0, 0, 0, 0);
            return;
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
            w[i][j] = __ldcs(reinterpret_cast<const uint4 *>(row + j * 64 + t * 16));
    }
    __device__ __forceinline__ void widen(uint32_t (&f)[D / 16][4]) const
    {
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[2 * j][i] = w[i][j].x;
                f[2 * j][2 + i] = w[i][j].y;
                f[2 * j + 1][i] = w[i][j].z;
                f[2 * j + 1][2 + i] = w[i][j].w;
            }
    }
};

template <int D>
struct Keys<MERCURY_ELEM_E4M3, D> {
    static constexpr int kRun = 16;
    static constexpr bool kF16 = true;
    static constexpr int kRowB = D;
    uint4 w[2][D / 64];
    __device__ __forceinline__ void load(int i, const char *row, int t)
    {
        if (!row) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                w[i][j] = make_uint4(0, 0, 0, 0);
            return;
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            w[i][j] = __ldcs(reinterpret_cast<const uint4 *>(row + j * 64 + t * 16));
    }
    __device__ __forceinline__ void widen(uint32_t (&f)[D / 16][4]) const
    {
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[4 * j + k][i] = e4m3_to_f16(x[k]);
                    f[4 * j + k][2 + i] = e4m3_to_f16(x[k] >> 16);
                }
            }
    }
};

template <int D>
struct Keys<MERCURY_ELEM_E2M1, D> {
    static constexpr int kRun = D / 8;
    static constexpr bool kF16 = true;
    static constexpr int kRowB = D / 2 + D / 16;
    uint32_t w[2][2][D / 64], s[2][D / 64];  // [key][run], all of a row's scales
    __device__ __forceinline__ void load(int i, const char *row, int t)
    {
        if (!row) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                w[i][0][j] = w[i][1][j] = s[i][j] = 0;
            return;
        }
        if constexpr (D == 128) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint2 x = *reinterpret_cast<const uint2 *>(row + j * 32 + t * 8);
                w[i][j][0] = x.x;
                w[i][j][1] = x.y;
            }
            const uint2 x = *reinterpret_cast<const uint2 *>(row + 64);
            s[i][0] = x.x;
            s[i][1] = x.y;
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[i][j][0] = *reinterpret_cast<const uint32_t *>(row + j * 16 + t * 4);
            s[i][0] = *reinterpret_cast<const uint32_t *>(row + 32);
        }
    }
    __device__ __forceinline__ void widen(uint32_t (&f)[D / 16][4]) const
    {
        // this lane's two runs' scales
        const int t = threadIdx.x & 3;
        const uint32_t pick = D == 128 ? t | (4 + t) << 4 : t / 2 | (2 + t / 2) << 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t both = e4m3_to_f16(__byte_perm(s[i][0], s[i][D / 64 - 1], pick));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t scale = __byte_perm(both, 0, j ? 0x3232 : 0x1010);
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const uint32_t x = w[i][j][k];
                    const int kk = j * (D / 32) + 2 * k;
                    f[kk][i] = mul_f16(e2m1_to_f16<0>(x), scale);
                    f[kk][2 + i] = mul_f16(e2m1_to_f16<1>(x), scale);
                    f[kk + 1][i] = mul_f16(e2m1_to_f16<2>(x), scale);
                    f[kk + 1][2 + i] = mul_f16(e2m1_to_f16<3>(x), scale);
                }
            }
        }
    }
};

// Tiles of sequence b.
__device__ __forceinline__ int mass_keys(const MassArgs &a, int b)
{
    return (int)min((long long)keys_of(a.p, b), a.width);
}

__device__ __forceinline__ int mass_tiles(const MassArgs &a, int b)
{
    return (mass_keys(a, b) + kMassTile - 1) / kMassTile;
}

template <bool M>
struct Masked {
    static constexpr bool value = M;
};

// Where a share's first tile lies.
struct Spot {
    int b, h, j;      // sequence, head, tile
    int keys, tiles;  // of the sequence
};

__device__ __forceinline__ void check_lengths(const MassArgs &a, int tid)
{
    if (blockIdx.x == 0 && a.r0 == 0)
        for (int b = tid; b < a.p.B; b += kMassThreads) {
            if (a.p.seq_lens[b] != mass_keys(a, b))
                record_bounds(0xb01);
            if (a.p.new_lens && a.p.new_lens[b] != new_of(a.p, b))
                record_bounds(0xb02);
        }
}

// The tiles of all heads in order, in equal shares: this block's are at .. end -
// 1, the first of them s.
__device__ __forceinline__ bool find_share(const MassArgs &a, int lane, Spot &s, long long &at, long long &end)
{
    const PagedArgs &p = a.p;
    long long total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        total += __reduce_add_sync(0xffffffffu, b < p.B ? mass_tiles(a, b) : 0);
    }
    total *= p.Hkv;
    at = total * blockIdx.x / gridDim.x;
    end = total * (blockIdx.x + 1) / gridDim.x;
    if (at >= end)
        return false;
    long long base = 0;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int mine = b < p.B ? mass_tiles(a, b) : 0;
        const int incl = warp_scan(mine, lane);
        const unsigned in = __ballot_sync(0xffffffffu, (base + incl) * p.Hkv > at);
        if (in) {
            const int l = __ffs(in) - 1;
            s.b = b0 + l;
            base += __shfl_sync(0xffffffffu, incl - mine, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    s.keys = mass_keys(a, s.b);
    s.tiles = mass_tiles(a, s.b);
    s.h = (int)((at - base * p.Hkv) / s.tiles);
    s.j = (int)(at - base * p.Hkv - (long long)s.h * s.tiles);
    return true;
}

// The tile behind x; there is one in the share.
__device__ __forceinline__ Spot next_spot(const MassArgs &a, Spot x)
{
    if (++x.j == x.tiles) {
        x.j = 0;
        if (++x.h == a.p.Hkv) {
            x.h = 0;
            do {
                ++x.b;
                x.keys = mass_keys(a, x.b);
                x.tiles = mass_tiles(a, x.b);
            } while (x.tiles == 0);
        }
    }
    return x;
}

// A row's constants.  mul (with mul_lo, what its rounding left out): from the
// product of the operands to log2 units; l: its lse.
__device__ __forceinline__ Row row_of(float mul, float mul_lo, float l, int step)
{
    constexpr float kLog2eLo = 1.9259629911266174e-8f;  // log2(e) less its nearest float
    const float nl = -l * kLog2e;
    const float off = mul == 0.f ? 0.f : mul_lo / mul;
    const float more = fmaf(-l, kLog2e, -nl) - l * kLog2eLo + l * kLog2e * off;  // what nl leaves out
    const bool counts = fabsf(l) < INFINITY || l != l;
    return Row{mul, counts ? nl : -INFINITY, counts ? exp2f(more) : 0.f, step};
}

// The power of two that brings `top` to [2^14, 2^15), and its inverse, both normal.
__device__ __forceinline__ void scale_of(float top, float &to, float &back)
{
    int up = 14 + 127 - (int)(__float_as_uint(top) >> 23);
    up = min(max(up, -110), 110);
    to = __uint_as_float((uint32_t)(127 + up) << 23);
    back = __uint_as_float((uint32_t)(127 - up) << 23);
}

// Blocks an SM: rows of 64 leave too few bytes on their way with two (one token
// of 8 sequences of 26K, 16 bits 46.7 us and with three 40.7, e4m3 40.9 and 36.0,
// e2m1 43.8 and 40.1; four spill: 48, 38, 49), rows of 128 spill with three.
constexpr int blocks_of(int D)
{
    return D == 64 ? 3 : 2;
}

template <int ELEM, int D>
__global__ void __launch_bounds__(kMassThreads, blocks_of(D)) attn_mass_kernel(const __grid_constant__ MassArgs a)
{
    using K = Keys<ELEM, D>;
    constexpr int KK = D / 16, RUN = K::kRun;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n_rt = (a.rows + 7) / 8;
    uint2 *const qs = reinterpret_cast<uint2 *>(smem);                       // [row tile][k-step][lane]
    Row *const rows = reinterpret_cast<Row *>(smem + n_rt * KK * 32 * 8);    // [row]
    const PagedArgs &p = a.p;
    const PagedView &c = p.cache;
    chain_wait();
    check_lengths(a, tid);
    Spot s;
    long long at, end;
    if (!find_share(a, lane, s, at, end))
        return;
    auto next_of = [&](const Spot &x) { return next_spot(a, x); };
    K keys;
    float prev = 0.f;  // of key g (t = 0) or g + 8 (t = 1)
    const bool one_page = c.page_size % 16 == 0;  // the 16 keys of a warp lie in one
    const long long page_bytes = c.page_stride * (ELEM == MERCURY_ELEM_BF16 ? 2 : 1), head_bytes = (long long)c.page_size * K::kRowB;
    auto load = [&](const Spot &x) {
        const int k0 = x.j * kMassTile + warp * 16;
        if (k0 >= x.keys)
            return;
        // (behind the last key: that key again, whose sum is not written)
        const int last = x.keys - 1 - k0;
        auto row_at = [&](int key) -> const char * {
            const int pg = page_of(c, key), page = c.table[x.b * c.table_stride + pg];
            if (page >= 0 && page < c.num_pages)
                return c.k + page * page_bytes + x.h * head_bytes + (key - pg * c.page_size) * (long long)K::kRowB;
            record_bounds(0xb03);  // such keys count as zeros
            return nullptr;
        };
        if (one_page) {
            const char *const row = row_at(k0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                keys.load(i, row ? row + min(g + 8 * i, last) * K::kRowB : nullptr, t);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                keys.load(i, row_at(k0 + min(g + 8 * i, last)), t);
        }
        const int key = k0 + g + 8 * t;
        prev = 0.f;
        if (a.mass && t < 2 && key < x.keys)
            prev = a.mass[((long long)x.b * p.Hkv + x.h) * a.width + key];
    };
    load(s);
    int job = -1, n_new = 0;
    for (;;) {
        const Spot now = s;
        const int this_job = now.b * p.Hkv + now.h;
        uint32_t f[KK][4];
        keys.widen(f);
        const float was = prev;
        const bool on = ++at < end;
        if (on) {
            s = next_of(now);
            load(s);  // on its way while this tile is computed
        }
        if (this_job != job) {
            // this head's queries
            job = this_job;
            n_new = new_of(p, now.b);
            __syncthreads();
            float ks = 1.f;
            if (K::kF16)
                ks = c.k_scale[now.h];
            for (int rt = warp; rt < n_rt; rt += kMassWarps) {
                const int r = a.r0 + rt * 8 + g;
                const int head = p.Sq == 1 ? r : r / p.Sq, i = r - head * p.Sq;
                const bool live = rt * 8 + g < a.rows && i < n_new;
                const __nv_bfloat16 *src = p.q + now.b * p.qs.b + (now.h * p.G + head) * p.qs.h + i * p.qs.s;
                uint2 q[KK];
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    q[kk] = live ? *reinterpret_cast<const uint2 *>(src + kk / (RUN / 4) * (4 * RUN) + t * RUN +
                                                                    kk % (RUN / 4) * 4)
                                 : make_uint2(0, 0);
                float mul = a.mul, mul_lo = a.mul_lo;  // to log2 units, of the product of the operands
                if constexpr (K::kF16) {
                    // to fp16, scaled by a power of two that brings the row's
                    // largest element to [2^14, 2^15): exact down to 2^-28 of it
                    float top = 0.f;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(q[kk].x)), fabsf(bf16_hi(q[kk].x))),
                                               fmaxf(fabsf(bf16_lo(q[kk].y)), fabsf(bf16_hi(q[kk].y)))));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    float to, back;
                    scale_of(top, to, back);
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        q[kk].x = pack_f16(bf16_lo(q[kk].x) * to, bf16_hi(q[kk].x) * to);
                        q[kk].y = pack_f16(bf16_lo(q[kk].y) * to, bf16_hi(q[kk].y) * to);
                    }
                    const float hi = a.mul * ks;
                    mul_lo = (fmaf(a.mul, ks, -hi) + a.mul_lo * ks) * back;
                    mul = hi * back;
                }
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    qs[(rt * KK + kk) * 32 + lane] = q[kk];
                if (t == 0) {
                    rows[rt * 8 + g] = row_of(mul, mul_lo, live ? a.lse[(long long)this_job * p.R + r] : INFINITY, i);
                }
            }
            __syncthreads();
        }
        const int k0 = now.j * kMassTile + warp * 16;
        const int seen_by_all = p.causal ? now.keys - n_new + 1 : now.keys;
        float sum[2] = {0.f, 0.f};
        auto add_rows = [&](auto masked) {
#pragma unroll 2
            for (int rt = 0; rt < n_rt; ++rt) {
                // in 2 sums of d/2 products each, added at the end
                float x[2][4];
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    const uint2 q = qs[(rt * KK + kk) * 32 + lane];
                    if (kk < 2)
                        mma_first<K::kF16>(x[kk], f[kk][0], f[kk][1], f[kk][2], f[kk][3], q.x, q.y);
                    else
                        mma<K::kF16>(x[kk & 1], f[kk][0], f[kk][1], f[kk][2], f[kk][3], q.x, q.y);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Row r = rows[rt * 8 + 2 * t + e];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float w = ex2_approx(fmaf(x[0][2 * i + e] + x[1][2 * i + e], r.mul, r.nl));
                        bool counts = r.rest != 0.f;  // (a product with 0 would let a key's infinity or NaN through)
                        if constexpr (decltype(masked)::value)
                            counts &= k0 + g + 8 * i < (p.causal ? seen_by_all + r.step : now.keys);
                        if (counts)
                            sum[i] = fmaf(w, r.rest, sum[i]);
                    }
                }
            }
        };
        if (k0 + 16 > seen_by_all) {
            if (k0 < now.keys)
                add_rows(Masked<true>());
        } else {
            add_rows(Masked<false>());
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        }
        const int key = k0 + g + 8 * t;
        if (t < 2 && key < now.keys)
            a.out[(long long)this_job * a.width + key] = was + (t ? sum[1] : sum[0]);
        if (!on)
            break;
    }
}

// Many rows: on the tensor unit.  A tile's 128 keys are M, the rows N (64, 128
// or 256 of a launch), and each of eight warps reads the scores of 32 keys and
// half of the rows back, a key a lane, so that a lane adds up its key's weights
// without any exchange.  Keys are widened to 16 bits on their way into shared
// memory; the product's time (128 rows: 256 cycles a tile) is a fraction of the
// exponentials' (512), and two blocks an SM overlap one's product and loads
// with the other's exponentials.  What a row costs there is its constants, read
// from shared memory by every warp: so there is only one (of four rows at a
// time), the exponent's summand; the factor is one for all rows, since their
// queries are scaled by one power of two, and what rounding the summand leaves
// out, 2^-24 of lse, is left out.  Such a scale rounds elements to 2^-40 of the
// largest of all rows.  So it is taken where no eight elements that lie together
// have a largest one 2^kApart below that one, but for zeros: they are rounded to
// 2^-27 of their own largest, far below what the sum of the products in 32 bits
// costs.  Else each row has a scale of its own and its factor is read too, so
// that no row's weights hang on another's queries.
template <int ELEM, int D>
struct Raw {  // half of a key's row
    static constexpr int kWords = ELEM == MERCURY_ELEM_BF16 ? D / 4 : ELEM == MERCURY_ELEM_E4M3 ? D / 8 : D / 16 + 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char *row, int half)
    {
        if (!row) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = 0;
            return;
        }
        if constexpr (ELEM == MERCURY_ELEM_E2M1) {
            // rows of 72 (36) bytes
#pragma unroll
            for (int i = 0; i < D / 16; i += D / 64) {
                const char *const from = row + half * (D / 4) + 4 * i;
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(from);
                    w[i] = x.x;
                    w[i + 1] = x.y;
                } else {
                    w[i] = *reinterpret_cast<const uint32_t *>(from);
                }
            }
            if constexpr (D == 128)
                w[kWords - 1] = *reinterpret_cast<const uint32_t *>(row + 64 + 4 * half);
            else
                w[kWords - 1] = *reinterpret_cast<const uint16_t *>(row + 32 + 2 * half);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(row + half * (kWords * 4) + 4 * i));
                w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
            }
        }
    }
    // elements 8 i .. + 7 as four words of the operand
    __device__ __forceinline__ void widen(int i, uint32_t (&o)[4]) const
    {
        if constexpr (ELEM == MERCURY_ELEM_BF16) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = w[4 * i + k];
        } else if constexpr (ELEM == MERCURY_ELEM_E4M3) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                o[2 * k] = e4m3_to_f16(w[2 * i + k]);
                o[2 * k + 1] = e4m3_to_f16(w[2 * i + k] >> 16);
            }
        } else {
            const uint32_t b = w[kWords - 1] >> (8 * (i / 2)) & 0xffu, scale = e4m3_to_f16(b | b << 8);
            o[0] = mul_f16(e2m1_to_f16<0>(w[i]), scale);
            o[1] = mul_f16(e2m1_to_f16<1>(w[i]), scale);
            o[2] = mul_f16(e2m1_to_f16<2>(w[i]), scale);
            o[3] = mul_f16(e2m1_to_f16<3>(w[i]), scale);
        }
    }
};

// Where 16-byte chunk c of a row lies in an operand of `rows` rows: column
// blocks of 64 elements, rows of 128 bytes, chunks permuted by the row (the
// 128-byte swizzle).
__device__ __forceinline__ int operand_at(int row, int c, int rows)
{
    return c / 8 * rows * 128 + row * 128 + ((c % 8 ^ (row & 7)) << 4);
}

constexpr int wide_smem(int D, int N)
{
    return 128 * D * 2 + N * D * 2 + N * 12 + 128 * 4 + 48;
}

constexpr int kApart = 12;

// Magnitudes of bf16 elements, as 16-bit integers, whose order is theirs: two's,
// infinite and NaN ones as zero.
__device__ __forceinline__ uint32_t magnitude(uint32_t w)
{
    w &= 0x7fff7fffu;
    return w & ~__vcmpgeu2(w, 0x7f807f80u);
}

// The largest of eight, in both halves.
__device__ __forceinline__ uint32_t top_of_eight(const uint4 &x)
{
    const uint32_t w = __vmaxu2(__vmaxu2(magnitude(x.x), magnitude(x.y)), __vmaxu2(magnitude(x.z), magnitude(x.w)));
    return __vmaxu2(w, __byte_perm(w, 0, 0x1032));
}

// The largest element of each of a head's rows of a launch that counts, a row a thread.
template <int D>
__device__ __forceinline__ void row_tops(const MassArgs &a, int b, int h, int n_new, float *tops)
{
    const PagedArgs &p = a.p;
    const int n = threadIdx.x, r = a.r0 + n, head = r / p.Sq, i = r - head * p.Sq;
    if (n >= a.wide)
        return;
    uint32_t top = 0;
    if (n < a.rows && i < n_new && fabsf(a.lse[((long long)b * p.Hkv + h) * p.R + r]) != INFINITY) {
        const uint4 *const src = reinterpret_cast<const uint4 *>(p.q + b * p.qs.b + (h * p.G + head) * p.qs.h + i * p.qs.s);
#pragma unroll 1
        for (int k = 0; k < D / 8; ++k)
            top = __vmaxu2(top, top_of_eight(src[k]));
    }
    tops[n] = __uint_as_float(top << 16);
}

template <int ELEM, int D>
__global__ void __launch_bounds__(kMassThreads, 2) attn_mass_wide_kernel(const __grid_constant__ MassArgs a)
{
    constexpr bool kF16 = ELEM != MERCURY_ELEM_BF16;
    constexpr int ROWB = ELEM == MERCURY_ELEM_BF16 ? 2 * D : ELEM == MERCURY_ELEM_E4M3 ? D : D / 2 + D / 16;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.wide;
    char *const keys_at = smem, *const queries_at = smem + 128 * D * 2;
    float *const summands = reinterpret_cast<float *>(queries_at + N * D * 2);  // -inf: the row counts nothing
    int *const steps = reinterpret_cast<int *>(summands + N);                   // of the new tokens
    float *const factors = reinterpret_cast<float *>(steps + N);                // from products to log2 units
    float *const halves = factors + N;
    uint64_t *const done = reinterpret_cast<uint64_t *>(halves + 128);
    uint32_t *const slot = reinterpret_cast<uint32_t *>(done + 1);
    // Each warp's of a job's queries (bf16's bits): the largest magnitude; in the upper
    // half the smallest of eight elements' largest, but for zeros, taken from infinity.
    uint32_t *const extremes = slot + 2;
    const PagedArgs &p = a.p;
    const PagedView &c = p.cache;
    chain_wait();
    check_lengths(a, tid);
    Spot now;
    long long at, end;
    if (!find_share(a, lane, now, at, end))
        return;
    if (tid == 0) {
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(slot, N);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;

    Raw<ELEM, D> raw;  // half (tid & 1) of key tid / 2
    float prev = 0.f;  // of key tid (the first 128 threads)
    // A tile's pages are asked for a tile before its keys are, and these a tile
    // before they are used.
    int page = -1;
    auto look_up = [&](const Spot &x) {
        const int key = x.j * kMassTile + tid / 2;
        if (key < x.keys)
            page = c.table[x.b * c.table_stride + page_of(c, key)];
    };
    auto load = [&](const Spot &x) {
        const int key = x.j * kMassTile + tid / 2;
        const char *row = nullptr;
        if (key < x.keys) {
            if (page >= 0 && page < c.num_pages)
                row = c.k + page * c.page_stride * (ELEM == MERCURY_ELEM_BF16 ? 2 : 1) +
                      ((long long)x.h * c.page_size + key - page_of(c, key) * c.page_size) * ROWB;
            else
                record_bounds(0xb03);  // such keys count as zeros
        }
        raw.load(row, tid & 1);
        const int mine = x.j * kMassTile + tid;
        prev = 0.f;
        if (a.mass && tid < 128 && mine < x.keys)
            prev = a.mass[((long long)x.b * p.Hkv + x.h) * a.width + mine];
    };
    look_up(now);
    load(now);
    Spot next = now;
    if (at + 1 < end) {
        next = next_spot(a, now);
        look_up(next);
    }
    uint32_t idesc = 0, parity = 0;
    if (N == 64)
        idesc = idesc_bf16_f32(128, 64, false);
    else if (N == 128)
        idesc = idesc_bf16_f32(128, 128, false);
    else
        idesc = idesc_bf16_f32(128, 256, false);
    if (kF16)
        idesc &= ~((1u << 7) | (1u << 10));  // both operands fp16
    int job = -1;
    float mul = a.mul;
    bool late = false;
    for (;;) {
        const int n_new = new_of(p, now.b);
        const int this_job = now.b * p.Hkv + now.h;
        if (this_job != job) {
            // this head's queries (the last product that read the others is done)
            job = this_job;
            // lanes of a row, rows at a time, loads on their way (16-bit keys, whose
            // next tile takes more registers: with 8 they spill, 128 rows 213 us)
            constexpr int LPR = D / 8, EACH = kMassThreads / LPR, U = kF16 ? 8 : 4;
            const int ch = tid % LPR;
            const __nv_bfloat16 *const head_q = p.q + now.b * p.qs.b + (now.h * p.G + a.head0) * p.qs.h;
            const float *const head_lse = a.lse + (long long)this_job * p.R;
            float mul_lo = a.mul_lo, to = 1.f;
            bool apart = false;
            mul = a.mul;
            uint4 x[U];
            // (n + step0 is below 384: exact)
            auto head_of = [&](int n) { return (n + a.step0) * a.per_sq >> 16; };
            // Rows' elements; their lse and new tokens go where the rows' constants
            // do.  Where all rows share a scale, one that counts nothing is taken as
            // zeros: the scale may not hang on what it holds (nor on an infinity).
            auto load_rows = [&](int n0) {
                float l[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int n = n0 + u * EACH, r = a.r0 + n, up = head_of(n), i = n + a.step0 - up * p.Sq;
                    x[u] = make_uint4(0, 0, 0, 0);
                    l[u] = INFINITY;
                    if (n < a.rows && i < n_new) {
                        x[u] = *reinterpret_cast<const uint4 *>(head_q + up * p.qs.h + i * p.qs.s + ch * 8);
                        if (kF16 || ch == 0)
                            l[u] = head_lse[r];
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int n = n0 + u * EACH;
                    if (kF16) {
                        const uint32_t keep = fabsf(l[u]) == INFINITY ? 0u : 0xffffffffu;
                        x[u].x &= keep, x[u].y &= keep, x[u].z &= keep, x[u].w &= keep;
                    }
                    if (ch == 0 && n < N) {
                        summands[n] = l[u];
                        steps[n] = n + a.step0 - head_of(n) * p.Sq;
                    }
                }
            };
            if constexpr (kF16) {
                uint32_t most = 0, few = 0xffffffffu;
                for (int n0 = tid / LPR; n0 < N; n0 += U * EACH) {
                    load_rows(n0);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint32_t top = top_of_eight(x[u]);
                        most = __vmaxu2(most, top);
                        few = __vminu2(few, __vsub2(top, 0x00010001u));  // (zero above all)
                    }
                }
                constexpr uint32_t kInf = 0x7f80;
                most = __reduce_max_sync(0xffffffffu, most & 0xffffu);
                few = kInf - min(__reduce_min_sync(0xffffffffu, few & 0xffffu) + 1, kInf);
                if (lane == 0)
                    extremes[warp] = most | few << 16;
                __syncthreads();
                {
                    const uint4 y = *reinterpret_cast<const uint4 *>(extremes), z = *reinterpret_cast<const uint4 *>(extremes + 4);
                    most = __vmaxu2(__vmaxu2(__vmaxu2(y.x, y.y), __vmaxu2(y.z, y.w)), __vmaxu2(__vmaxu2(z.x, z.y), __vmaxu2(z.z, z.w)));
                }
                few = most >> 16;
                apart = few != 0 && (int)((most & 0xffffu) >> 7) - (int)((kInf - few) >> 7) > kApart;
                if (apart) {
                    row_tops<D>(a, now.b, now.h, n_new, factors);
                    __syncthreads();
                }
                float back;
                scale_of(__uint_as_float(most << 16), to, back);
                const float ks = c.k_scale[now.h], hi = a.mul * ks;
                if (apart)
                    back = 1.f;
                mul_lo = (fmaf(a.mul, ks, -hi) + a.mul_lo * ks) * back;
                mul = hi * back;
            }
            for (int n0 = tid / LPR; n0 < N; n0 += U * EACH) {
                if (!kF16 || N > U * EACH)  // (else they are here)
                    load_rows(n0);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int n = n0 + u * EACH;
                    if (n >= N)
                        break;
                    float back = 1.f;
                    if (kF16 && apart) {
                        scale_of(factors[n], to, back);
                        __syncwarp();  // (the row's lanes have read it)
                    }
                    if (kF16)
                        x[u] = make_uint4(pack_f16(bf16_lo(x[u].x) * to, bf16_hi(x[u].x) * to), pack_f16(bf16_lo(x[u].y) * to, bf16_hi(x[u].y) * to),
                                          pack_f16(bf16_lo(x[u].z) * to, bf16_hi(x[u].z) * to), pack_f16(bf16_lo(x[u].w) * to, bf16_hi(x[u].w) * to));
                    *reinterpret_cast<uint4 *>(queries_at + operand_at(n, ch, N)) = x[u];
                    if (ch == 0) {
                        // (of mul and lse in log2 units, as in row_of)
                        factors[n] = mul * back;
                        const float off = mul == 0.f ? 0.f : mul_lo / mul, l = summands[n];
                        summands[n] = fabsf(l) < INFINITY || l != l ? fmaf(-l, kLog2e, l * kLog2e * off) : -INFINITY;
                    }
                }
            }
            // (the short way's sums are not finite then, and made again by the rows' factors)
            if (apart)
                mul = __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t o[4];
            raw.widen(i, o);
            *reinterpret_cast<uint4 *>(keys_at + operand_at(tid / 2, (tid & 1) * (D / 16) + i, 128)) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
        const float was = prev;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            const uint32_t leader = elect_lane();
            const uint64_t dk = smem_desc_sw128(smem_u32(keys_at), 16, 1024), dq = smem_desc_sw128(smem_u32(queries_at), 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_ss_w(tmem, dk + (uint32_t)((kk / 4 * 128 * 128 + kk % 4 * 32) >> 4),
                          dq + (uint32_t)((kk / 4 * N * 128 + kk % 4 * 32) >> 4), idesc, kk > 0 ? 1u : 0u, leader);
            if (!p.fault)  // (the test hook: the product's end is never told)
                umma_commit_w(done, leader);
        }
        const Spot tile = now;
        const bool on = ++at < end;
        if (on) {
            now = next;
            load(now);  // on its way while this tile is computed
            if (at + 1 < end) {
                next = next_spot(a, now);
                look_up(next);
            }
        }
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(done, parity))
            if (globaltimer_ns() - t0 > p.wait_ns) {
                late = true;
                break;
            }
        parity ^= 1;
        tc_fence_after();
        const int k0 = tile.j * kMassTile, quarter = warp & 3, half = warp >> 2;
        const int key = k0 + quarter * 32 + lane;
        const int seen_by_all = p.causal ? tile.keys - n_new + 1 : tile.keys;
        float sum = 0.f;
        auto add_rows = [&](auto masked) {
            sum = 0.f;
            for (int n = half * (N / 2); n < half * (N / 2) + N / 2; n += 32) {
                uint32_t x[32];
                tmem_ld_x32(tmem + ((uint32_t)(quarter * 32) << 16) + n, x);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(summands + n + k);
                    const float nl[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = ex2_approx(fmaf(__uint_as_float(x[k + e]), kF16 && decltype(masked)::value ? factors[n + k + e] : mul, nl[e]));
                        if constexpr (decltype(masked)::value) {
                            if (nl[e] != -INFINITY && key < (p.causal ? seen_by_all + steps[n + k + e] : tile.keys))
                                sum += w;
                        } else {
                            sum += w;
                        }
                    }
                }
            }
        };
        // (An infinite or NaN key gives NaN in rows that count nothing, too: such
        // sums are made again, row by row; so are all where the rows have scales of
        // their own.)
        bool all = k0 + kMassTile > seen_by_all;
        if (!all) {
            add_rows(Masked<false>());
            all = __any_sync(0xffffffffu, !(fabsf(sum) < INFINITY));
        }
        if (all)
            add_rows(Masked<true>());
        if (half)
            halves[tid - 128] = sum;
        tc_fence_before();
        late = __syncthreads_or(late);
        if (late)
            break;
        if (!half && key < tile.keys)
            a.out[(long long)this_job * a.width + key] = was + (sum + halves[tid]);
        if (!on)
            break;
    }
    if (late) {
        if (tid == 0) {
            atomicOr(&g_paged_err_word, kErrTimeout);
            atomicCAS(&g_paged_err_site, 0u, 0xb04u);
        }
        // the product may still be on its way: its memory is given up once it
        // has ended, waited for with a limit too
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(done, parity ^ 1) && globaltimer_ns() - t0 <= p.wait_ns)
            ;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, N);
    }
}

template <int ELEM, int D>
int launch(MassArgs &a, cudaStream_t stream, char *msg, size_t msg_len)
{
    auto *kernel = attn_mass_kernel<ELEM, D>;
    constexpr int kRowSmem = D / 16 * 4 * 8 + (int)sizeof(Row);
    KernelInfo ki;
    int rc = prepare_kernel((const void *)kernel, kMassRows * kRowSmem, &ki, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    KernelInfo wi;
    auto *wide_kernel = attn_mass_wide_kernel<ELEM, D>;
    rc = prepare_kernel((const void *)wide_kernel, wide_smem(D, kWideRows), &wi, msg, msg_len);
    if (rc != MERCURY_OK)
        return rc;
    const long long keys = (long long)a.p.cache.max_pages * a.p.cache.page_size;
    const long long most = ((keys < a.width ? keys : a.width) + kMassTile - 1) / kMassTile * a.p.B * a.p.Hkv;
    // On the tensor unit a tile takes the same time up to 64 rows; there it pays
    // from some 50 on where keys are narrow and each block has many tiles (8 x 8
    // heads, 32K, 64 rows by warps and on the tensor unit: d 64 16 bits 101 us and
    // 82, e4m3 87 and 78, e2m1 95 and 82; d 128 e2m1 130 and 103, 16 bits 149 and
    // 170, and e4m3 128 and 110, which goes by warps yet; 48 rows: d 64 16 bits 87
    // and 82, e4m3 75 and 78, d 128 e2m1 110 and 103; 2K tiles, d 64 e4m3, 64 rows:
    // 16.8 and 19.4; one sequence of 4K, d 128, 64 rows: 6.7 and 9.0).  More rows are
    // two launches by warps: one sequence of 4K, d 128, 68 rows 11.4 us and 10.2,
    // 128 rows 13.4 and 10.7, in 4 bits 10.9 and 10.8, 12.7 and 11.1; 128 rows of 8
    // x 20K to 32K 246 and 157, in 4 bits 215 and 107.
    const bool narrow_keys = D == 64 || ELEM == MERCURY_ELEM_E2M1;
    const bool wide = a.p.R > kMassRows || (a.p.R > 48 && narrow_keys && most >= 24LL * ki.sms);
    const int each = wide ? kWideRows : kMassRows;
    for (long long r0 = 0; r0 < a.p.R; r0 += each) {
        a.r0 = (int)r0;
        a.head0 = a.r0 / a.p.Sq;
        a.step0 = a.r0 % a.p.Sq;
        a.rows = a.p.R - a.r0 < each ? a.p.R - a.r0 : each;
        a.wide = !wide ? 0 : a.rows <= 64 ? 64 : a.rows <= 128 ? 128 : 256;
        const int smem = wide ? wide_smem(D, a.wide) : (a.rows + 7) / 8 * 8 * kRowSmem;
        const int per_sm = wide ? 2 : blocks_of(D);
        const long long grid = most < (long long)ki.sms * per_sm ? most : (long long)ki.sms * per_sm;
        const cudaError_t e = launch_chained(wide ? wide_kernel : kernel, dim3((unsigned)grid), kMassThreads, smem, stream, a);
        if (e != cudaSuccess) {
            snprintf(msg, msg_len, "attention weight launch: %s", cudaGetErrorString(e));
            return MERCURY_ECUDA;
        }
        a.mass = a.out;  // further rows are added to what the first ones gave
    }
    return MERCURY_OK;
}

template <int D>
int launch_elem(MassArgs &a, int elem, cudaStream_t stream, char *msg, size_t msg_len)
{
    return elem == MERCURY_ELEM_BF16   ? launch<MERCURY_ELEM_BF16, D>(a, stream, msg, msg_len)
           : elem == MERCURY_ELEM_E4M3 ? launch<MERCURY_ELEM_E4M3, D>(a, stream, msg, msg_len)
                                       : launch<MERCURY_ELEM_E2M1, D>(a, stream, msg, msg_len);
}

}  // namespace

int launch_attn_mass(const void *q, const Strides &qs, const mercury_paged_cache &cache, const int *seq_lens,
                     const int *new_lens, int B, int Hq, int Sq, int causal, const float *lse, const float *mass,
                     float *out, long long width, unsigned long long wait_ns, int fault, cudaStream_t stream, char *msg,
                     size_t msg_len)
{
    MassArgs a = {};
    a.p = paged_args(q, qs, cache, seq_lens, new_lens, B, Hq, Sq, causal, nullptr, nullptr, 0, wait_ns, fault);
    a.lse = lse;
    a.mass = mass;
    a.out = out;
    a.width = width;
    a.per_sq = ((1 << 16) + Sq - 1) / Sq;
    const double mul = 1.4426950408889634074 / sqrt((double)cache.d);
    a.mul = (float)mul;
    a.mul_lo = (float)(mul - (double)a.mul);
    return cache.d == 128 ? launch_elem<128>(a, cache.elem, stream, msg, msg_len)
                          : launch_elem<64>(a, cache.elem, stream, msg, msg_len);
}

int read_and_clear_mass_error(unsigned int *word, unsigned int *site, char *msg, size_t msg_len)
{
    return read_and_clear_words(g_paged_err_word, g_paged_err_site, "attention weight", word, site, msg, msg_len);
}

}  // namespace mercury
