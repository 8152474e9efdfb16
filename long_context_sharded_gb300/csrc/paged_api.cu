// paged_api.cu -- the C ABI of the serving operators: rotary plans (host
// code), and the validation and dispatch of the rotation, the cache append and
// paged attention.  Contracts are in include/mercury_attn.h.
#include <cuda_runtime.h>

#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "paged.cuh"

using namespace mercury;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool aligned(const void *p, uintptr_t a)
{
    return ((uintptr_t)p % a) == 0;
}

// The strides the caller gave, or those of a contiguous [B, H, S, d] tensor.
int read_strides(const long long *given, int H, int S, int d, const char *what, Strides *out)
{
    if (!given) {
        *out = Strides{(long long)H * S * d, (long long)S * d, d};
        return MERCURY_OK;
    }
    *out = Strides{given[0], given[1], given[2]};
    if (given[0] < 0 || given[1] < 0 || given[2] < 0)
        return set_error(MERCURY_EINVAL, "%s strides must be >= 0", what);
    return MERCURY_OK;
}

// Offsets of a strided [B, H, S, d] tensor stay below 2^62 elements.
int check_extent(const Strides &s, int B, int H, int S, const char *what)
{
    const double e = (double)s.b * (B - 1) + (double)s.h * (H - 1) + (double)s.s * (S - 1);
    if (e > 4.6e18)
        return set_error(MERCURY_EINVAL, "%s sizes overflow", what);
    return MERCURY_OK;
}

// An output's rows may not overlap: each stride steps over the extent of
// every smaller one (an axis of size 1 does not step).
int check_distinct(const Strides &s, int B, int H, int S, int d, const char *what)
{
    long long st[3] = {s.b, s.h, s.s};
    int n[3] = {B, H, S};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const long long a = st[i];
                st[i] = st[j];
                st[j] = a;
                const int b = n[i];
                n[i] = n[j];
                n[j] = b;
            }
    long long extent = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1)
            continue;
        if (st[i] < extent)
            return set_error(MERCURY_EINVAL, "%s rows overlap (strides %lld, %lld, %lld)", what, s.b, s.h, s.s);
        extent += st[i] * (n[i] - 1);
    }
    return MERCURY_OK;
}

int check_plan(const mercury_rope_plan *p, int d)
{
    if (p->rot_dim < 2 || p->rot_dim > MERCURY_MAX_ROT || p->rot_dim % 2 != 0)
        return set_error(MERCURY_EINVAL, "rope plan: rot_dim must be even, 2..%d (got %d)", MERCURY_MAX_ROT,
                         p->rot_dim);
    if (p->rot_dim > d)
        return set_error(MERCURY_EINVAL, "rope plan: rot_dim (%d) exceeds the head dim (%d)", p->rot_dim, d);
    return MERCURY_OK;
}

int check_cache(const mercury_paged_cache *c, int B)
{
    if (!c)
        return set_error(MERCURY_EINVAL, "cache is NULL");
    if (!c->k || !c->v || !c->block_table)
        return set_error(MERCURY_EINVAL, "cache: null pointer");
    if (c->elem != MERCURY_ELEM_BF16 && c->elem != MERCURY_ELEM_E4M3 && c->elem != MERCURY_ELEM_E2M1)
        return set_error(MERCURY_EINVAL, "cache: elem must be BF16, E4M3 or E2M1 (got %d)", c->elem);
    if (c->elem != MERCURY_ELEM_BF16 && (!c->k_scale || !c->v_scale))
        return set_error(MERCURY_EINVAL, "cache: an E4M3 or E2M1 cache needs k_scale and v_scale");
    if (c->d != 64 && c->d != 128)
        return set_error(MERCURY_EINVAL, "head dim must be 64 or 128 (got %d)", c->d);
    if (c->Hkv < 1 || c->page_size < 1 || c->num_pages < 1 || c->max_pages < 1 || c->B < 1)
        return set_error(MERCURY_EINVAL, "cache: Hkv, page_size, num_pages, max_pages and B must be >= 1");
    if (c->B != B)
        return set_error(MERCURY_EINVAL, "B (%d) does not match the cache's %d sequences", B, c->B);
    if (c->Hkv > 16384)
        return set_error(MERCURY_EINVAL, "Hkv must be at most 16384 (got %d)", c->Hkv);
    if ((long long)c->max_pages * c->page_size > (1LL << 30))
        return set_error(MERCURY_EINVAL, "max_pages * page_size must be at most 2^30 (got %lld)",
                         (long long)c->max_pages * c->page_size);
    // of a row: elements, or an E2M1 cache's bytes
    const int row = c->elem == MERCURY_ELEM_E2M1 ? c->d / 2 + c->d / 16 : c->d;
    if (c->elem == MERCURY_ELEM_E2M1 && c->page_size % 8 != 0)
        return set_error(MERCURY_EINVAL, "cache: an E2M1 cache's page_size must be a multiple of 8 (got %d)", c->page_size);
    if ((double)c->Hkv * c->page_size * row > 4.6e18 || c->page_stride < (long long)c->Hkv * c->page_size * row ||
        (double)c->page_stride * c->num_pages > 2.3e18)
        return set_error(MERCURY_EINVAL, "cache: page_stride %lld is less than a page, or sizes overflow",
                         c->page_stride);
    if (c->table_stride < c->max_pages)
        return set_error(MERCURY_EINVAL, "cache: table_stride (%lld) is less than max_pages (%d)", c->table_stride,
                         c->max_pages);
    const int es = c->elem == MERCURY_ELEM_BF16 ? 2 : 1;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride * es % 16 != 0)
        return set_error(MERCURY_EALIGN, "cache: k and v must be 16-byte aligned and pages multiples of 16 bytes apart");
    if (!aligned(c->block_table, 4) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return set_error(MERCURY_EALIGN, "cache: block_table and scales must be 4-byte aligned");
    return MERCURY_OK;
}

// What every call over a cache with queries [B, Hq, Sq, d] asks of them.
int check_queries(const void *q, const long long *q_strides, const mercury_paged_cache *cache, const int *seq_lens,
                  const int *new_lens, int B, int Hq, int Sq, Strides *qs)
{
    int rc = check_cache(cache, B);
    if (rc)
        return rc;
    if (Hq < 1 || Hq % cache->Hkv != 0)
        return set_error(MERCURY_EINVAL, "Hq (%d) must be a multiple of Hkv (%d)", Hq, cache->Hkv);
    if (Sq < 1 || Sq > 64)
        return set_error(MERCURY_EINVAL, "Sq must be in [1, 64] (got %d): longer prompts are mercury_attn_sharded's",
                         Sq);
    if ((double)B * Hq * Sq > (double)INT_MAX)
        return set_error(MERCURY_EINVAL, "B*Hq*Sq exceeds 2^31");
    rc = read_strides(q_strides, Hq, Sq, cache->d, "q", qs);
    if (rc == MERCURY_OK)
        rc = check_extent(*qs, B, Hq, Sq, "q");
    if (rc)
        return rc;
    if (!aligned(q, 16) || qs->b % 8 != 0 || qs->h % 8 != 0 || qs->s % 8 != 0)
        return set_error(MERCURY_EALIGN, "q must be 16-byte aligned, with strides of multiples of 8 elements");
    if (!aligned(seq_lens, 4) || !aligned(new_lens, 4))
        return set_error(MERCURY_EALIGN, "seq_lens and new_lens must be 4-byte aligned");
    return MERCURY_OK;
}

int attn_paged(const void *q, const long long *q_strides, const mercury_paged_cache *cache, const int *seq_lens,
               const int *new_lens, int B, int Hq, int Sq, int causal, void *out, float *lse, int out_bf16,
               void *stream)
{
    if (!q || !seq_lens || !out || !lse)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    Strides qs;
    int rc = check_queries(q, q_strides, cache, seq_lens, new_lens, B, Hq, Sq, &qs);
    if (rc)
        return rc;
    if (!aligned(out, 16))
        return set_error(MERCURY_EALIGN, "out must be 16-byte aligned");
    if (!aligned(lse, 4))
        return set_error(MERCURY_EALIGN, "lse must be 4-byte aligned");
    size_t len;
    char *msg = error_buffer(&len);
    cudaStream_t s = (cudaStream_t)stream;
    auto *launch = cache->elem == MERCURY_ELEM_E2M1 ? launch_attn_paged4 : launch_attn_paged;
    rc = launch(q, qs, *cache, seq_lens, new_lens, B, Hq, Sq, causal ? 1 : 0, out, lse, out_bf16, device_wait_ns(),
                paged_fault(), s, msg, len);
    return finish_call(rc, s);
}

}  // namespace

extern "C" {

int mercury_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_length,
                             double beta_fast, double beta_slow, double *freq, double *magnitude)
{
    if (!freq || !magnitude)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    if (rot_dim < 2 || rot_dim > MERCURY_MAX_ROT || rot_dim % 2 != 0)
        return set_error(MERCURY_EINVAL, "rot_dim must be even, 2..%d (got %d)", MERCURY_MAX_ROT, rot_dim);
    if (!(base > 1.0) || !isfinite(base))
        return set_error(MERCURY_EINVAL, "base must be finite and > 1");
    if (scaling < MERCURY_ROPE_NONE || scaling > MERCURY_ROPE_YARN)
        return set_error(MERCURY_EINVAL, "unknown frequency scaling %d", scaling);
    if (!(factor >= 1.0) || !isfinite(factor))
        return set_error(MERCURY_EINVAL, "factor must be finite and >= 1");
    if (scaling == MERCURY_ROPE_NTK && rot_dim < 4)
        return set_error(MERCURY_EINVAL, "the NTK scaling needs rot_dim >= 4");
    if (scaling == MERCURY_ROPE_YARN && (!(original_length > 0.0) || !isfinite(original_length) ||
                                         !(beta_slow >= 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast)))
        return set_error(MERCURY_EINVAL, "the YARN scaling needs original_length > 0 and beta_fast > beta_slow >= 0");
    if (scaling == MERCURY_ROPE_NTK)
        base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == MERCURY_ROPE_LINEAR)
            f /= factor;
        if (scaling == MERCURY_ROPE_YARN) {
            double g = (original_length * f / kTwoPi - beta_slow) / (beta_fast - beta_slow);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = g * f + (1.0 - g) * f / factor;
        }
        freq[i] = f;
    }
    *magnitude = scaling == MERCURY_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    return clear_error();
}

int mercury_rope_init(int rot_dim, int interleaved, const double *freq, double magnitude, mercury_rope_plan *plan)
{
    if (!freq || !plan)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    if (rot_dim < 2 || rot_dim > MERCURY_MAX_ROT || rot_dim % 2 != 0)
        return set_error(MERCURY_EINVAL, "rot_dim must be even, 2..%d (got %d)", MERCURY_MAX_ROT, rot_dim);
    if (!isfinite((float)magnitude))
        return set_error(MERCURY_EINVAL, "magnitude must be finite");
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!(freq[i] >= 0.0) || freq[i] > 1048576.0)
            return set_error(MERCURY_EINVAL, "freq[%d] must be in [0, 2^20]", i);
    plan->rot_dim = rot_dim;
    plan->interleaved = interleaved ? 1 : 0;
    plan->magnitude = (float)magnitude;
    for (int i = 0; i < MERCURY_MAX_ROT / 2; ++i) {
        // the fraction of a turn, exact as a multiple of 2^-64 for any
        // frequency above 2^-11 turns a position and to 2^-65 below
        double t = 0.0;
        if (i < rot_dim / 2) {
            t = freq[i] / kTwoPi;
            t = ldexp(t - floor(t), 64);
        }
        plan->turns[i] = (unsigned long long)t;
    }
    return clear_error();
}

int mercury_rope(const void *x, const long long *x_strides, const int *positions, long long pos_stride,
                 long long start, int B, int H, int S, int d, int elem, const mercury_rope_plan *plan, int inverse,
                 void *out, const long long *out_strides, void *stream)
{
    CallRange range(__func__);
    if (!x || !out || !plan)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    if (B < 1 || H < 1 || S < 1)
        return set_error(MERCURY_EINVAL, "B, H, S must be >= 1");
    if (H > 65535 || (long long)B * S > INT_MAX)
        return set_error(MERCURY_EINVAL, "H must be at most 65535 and B*S below 2^31");
    if (elem != MERCURY_ELEM_BF16 && elem != MERCURY_ELEM_FP32)
        return set_error(MERCURY_EINVAL, "elem must be BF16 or FP32 (got %d)", elem);
    if (d < 1 || d > 512)
        return set_error(MERCURY_EINVAL, "head dim must be in [1, 512] (got %d)", d);
    if (pos_stride < 0)
        return set_error(MERCURY_EINVAL, "pos_stride must be >= 0");
    int rc = check_plan(plan, d);
    Strides xs, os;
    if (rc == MERCURY_OK)
        rc = read_strides(x_strides, H, S, d, "x", &xs);
    if (rc == MERCURY_OK)
        rc = read_strides(out_strides, H, S, d, "out", &os);
    if (rc == MERCURY_OK)
        rc = check_extent(xs, B, H, S, "x");
    if (rc == MERCURY_OK)
        rc = check_extent(os, B, H, S, "out");
    if (rc == MERCURY_OK)
        rc = check_distinct(os, B, H, S, d, "out");
    if (rc)
        return rc;
    const int es = elem == MERCURY_ELEM_FP32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(out, es) || !aligned(positions, 4))
        return set_error(MERCURY_EALIGN, "x, out and positions must be aligned to their elements");
    int sms = 0;
    rc = device_sm_count(&sms);
    if (rc)
        return rc;
    size_t len;
    char *msg = error_buffer(&len);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_rope(x, xs, positions, pos_stride, start, B, H, S, d, elem, *plan, inverse, out, os, sms, s, msg, len);
    return finish_call(rc, s);
}

int mercury_kv_append(const void *k, const long long *k_strides, const void *v, const long long *v_strides, int B,
                      int S, const mercury_paged_cache *cache, const int *past_lens, const int *new_lens,
                      const mercury_rope_plan *rope, const void *q, const long long *q_strides, int Hq, void *q_out,
                      const long long *q_out_strides, void *stream)
{
    CallRange range(__func__);
    if (!k || !v || !past_lens || (q && !q_out))
        return set_error(MERCURY_EINVAL, "null pointer argument");
    int rc = check_cache(cache, B);
    if (rc)
        return rc;
    if (S < 1 || (long long)B * S > INT_MAX)
        return set_error(MERCURY_EINVAL, "S must be >= 1 and B*S below 2^31");
    if (q && (Hq < 1 || Hq > 32767))
        return set_error(MERCURY_EINVAL, "Hq must be in [1, 32767] (got %d)", Hq);
    const int d = cache->d, Hkv = cache->Hkv;
    Strides ks, vs, qs = {0, 0, 0}, os = {0, 0, 0};
    rc = read_strides(k_strides, Hkv, S, d, "k", &ks);
    if (rc == MERCURY_OK)
        rc = read_strides(v_strides, Hkv, S, d, "v", &vs);
    if (rc == MERCURY_OK)
        rc = check_extent(ks, B, Hkv, S, "k");
    if (rc == MERCURY_OK)
        rc = check_extent(vs, B, Hkv, S, "v");
    if (q) {
        if (rc == MERCURY_OK)
            rc = read_strides(q_strides, Hq, S, d, "q", &qs);
        if (rc == MERCURY_OK)
            rc = read_strides(q_out_strides, Hq, S, d, "q_out", &os);
        if (rc == MERCURY_OK)
            rc = check_extent(qs, B, Hq, S, "q");
        if (rc == MERCURY_OK)
            rc = check_extent(os, B, Hq, S, "q_out");
        if (rc == MERCURY_OK)
            rc = check_distinct(os, B, Hq, S, d, "q_out");
    }
    if (rc == MERCURY_OK && rope)
        rc = check_plan(rope, d);
    if (rc)
        return rc;
    if (!aligned(k, 2) || !aligned(v, 2) || !aligned(q, 2) || !aligned(q_out, 2) || !aligned(past_lens, 4) ||
        !aligned(new_lens, 4))
        return set_error(MERCURY_EALIGN, "k, v, q, q_out, past_lens and new_lens must be aligned to their elements");
    int sms = 0;
    rc = device_sm_count(&sms);
    if (rc)
        return rc;
    size_t len;
    char *msg = error_buffer(&len);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_kv_append(k, ks, v, vs, q, qs, q_out, os, *cache, past_lens, new_lens, B, Hq, S, rope, sms, s, msg,
                          len);
    return finish_call(rc, s);
}

int mercury_attn_paged(const void *q, const long long *q_strides, const mercury_paged_cache *cache,
                       const int *seq_lens, const int *new_lens, int B, int Hq, int Sq, int causal, float *out,
                       float *lse, void *stream)
{
    CallRange range(__func__);
    return attn_paged(q, q_strides, cache, seq_lens, new_lens, B, Hq, Sq, causal, out, lse, 0, stream);
}

int mercury_attn_paged_bf16(const void *q, const long long *q_strides, const mercury_paged_cache *cache,
                            const int *seq_lens, const int *new_lens, int B, int Hq, int Sq, int causal, void *out,
                            float *lse, void *stream)
{
    CallRange range(__func__);
    return attn_paged(q, q_strides, cache, seq_lens, new_lens, B, Hq, Sq, causal, out, lse, 1, stream);
}

int mercury_attn_paged_mass(const void *q, const long long *q_strides, const mercury_paged_cache *cache,
                            const int *seq_lens, const int *new_lens, int B, int Hq, int Sq, int causal,
                            const float *lse, const float *mass, float *out, long long width, void *stream)
{
    CallRange range(__func__);
    if (!q || !seq_lens || !lse || !out)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    Strides qs;
    int rc = check_queries(q, q_strides, cache, seq_lens, new_lens, B, Hq, Sq, &qs);
    if (rc)
        return rc;
    if (width < 1 || (double)width * B * cache->Hkv > 4.6e18)
        return set_error(MERCURY_EINVAL, "width must be >= 1, and B * Hkv * width below 2^62 (got %lld)", width);
    if (!aligned(lse, 4) || !aligned(mass, 4) || !aligned(out, 4))
        return set_error(MERCURY_EALIGN, "lse, mass and out must be 4-byte aligned");
    size_t len;
    char *msg = error_buffer(&len);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_attn_mass(q, qs, *cache, seq_lens, new_lens, B, Hq, Sq, causal ? 1 : 0, lse, mass, out, width,
                          device_wait_ns(), paged_fault(), s, msg, len);
    return finish_call(rc, s);
}

int mercury_kv_evict(const mercury_paged_cache *cache, const mercury_paged_cache *into, const float *mass,
                     long long width, const int *seq_lens, int B, int keep, int first, int last, int *out_lens,
                     int *kept, float *out_mass, long long out_width, void *stream)
{
    CallRange range(__func__);
    if (!mass || !seq_lens || !out_lens || !kept)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    int rc = check_cache(cache, B);
    if (rc == MERCURY_OK)
        rc = check_cache(into, B);
    if (rc)
        return rc;
    if (into->elem != cache->elem || into->Hkv != cache->Hkv || into->d != cache->d)
        return set_error(MERCURY_EINVAL, "both caches must have the same elem, Hkv and d");
    if (keep < 1 || first < 0 || last < 0 || (long long)first + last > keep)
        return set_error(MERCURY_EINVAL, "keep must be >= 1 and first and last >= 0, together at most keep (got %d, %d, %d)",
                         keep, first, last);
    if (keep > (long long)into->max_pages * into->page_size)
        return set_error(MERCURY_EINVAL, "keep (%d) exceeds the shorter cache's table (%lld)", keep,
                         (long long)into->max_pages * into->page_size);
    if (width < 1 || (double)width * B * cache->Hkv > 4.6e18)
        return set_error(MERCURY_EINVAL, "width must be >= 1, and B * Hkv * width below 2^62 (got %lld)", width);
    if (out_mass && (out_width < keep || (double)out_width * B * cache->Hkv > 4.6e18))
        return set_error(MERCURY_EINVAL, "out_width must be at least keep, and B * Hkv * out_width below 2^62 (got %lld)",
                         out_width);
    if (out_lens == seq_lens || (out_mass && out_mass == mass))
        return set_error(MERCURY_EINVAL, "out_lens and out_mass may not be seq_lens and mass");
    if (!aligned(mass, 4) || !aligned(seq_lens, 4) || !aligned(out_lens, 4) || !aligned(kept, 4) || !aligned(out_mass, 4))
        return set_error(MERCURY_EALIGN, "mass, seq_lens, out_lens, kept and out_mass must be 4-byte aligned");
    // (rows would be stored where others have yet to be read)
    if (into->block_table == cache->block_table && (into->k == cache->k || into->v == cache->v))
        return set_error(MERCURY_EINVAL, "a sequence cannot be shortened within its own pages");
    size_t len;
    char *msg = error_buffer(&len);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_kv_evict(*cache, *into, mass, width, seq_lens, keep, first, last, out_lens, kept, out_mass, out_width, s,
                         msg, len);
    return finish_call(rc, s);
}

int mercury_kv_read(const mercury_paged_cache *cache, const int *seq_lens, int B, int S, void *k_out, void *v_out,
                    void *stream)
{
    CallRange range(__func__);
    if (!seq_lens || !k_out || !v_out)
        return set_error(MERCURY_EINVAL, "null pointer argument");
    int rc = check_cache(cache, B);
    if (rc)
        return rc;
    if (S < 1)
        return set_error(MERCURY_EINVAL, "S must be >= 1 (got %d)", S);
    if (!aligned(k_out, 16) || !aligned(v_out, 16))
        return set_error(MERCURY_EALIGN, "k_out and v_out must be 16-byte aligned");
    if (!aligned(seq_lens, 4))
        return set_error(MERCURY_EALIGN, "seq_lens must be 4-byte aligned");
    if (k_out == v_out)
        return set_error(MERCURY_EINVAL, "k_out and v_out must be two tensors");
    size_t len;
    char *msg = error_buffer(&len);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_kv_read(*cache, seq_lens, S, k_out, v_out, s, msg, len);
    return finish_call(rc, s);
}

}  // extern "C"
