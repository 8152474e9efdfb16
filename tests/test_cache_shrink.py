"""A cache of 4 bits, attention weights of cached keys, eviction by them and a
cache read back, against their definitions in 64 bits.

Bounds.  4-bit rows: none, the codes are those of the real quotients; with a
rotation the reference computes them in 64 bits, whose own error (1e-15 of a
value) reaches a border between two codes for no input here.  Attention: as in
test_paged.py; a 4-bit element times its block's scale is exact in fp16.
Weights: a score is a sum of d products in a 32-bit accumulator (2^-21 of the
sum of their magnitudes over sqrt(d)); the exponent's factors and sums round a
few times, 2^-22 of |score| + |lse|; 2^exponent is good to 2^-21; R weights added
one after another lose R 2^-24 of their sum, and what they are added to 2^-23.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests.test_paged import (  # noqa: F401
    BF16, E4M3, FP32, SHAPES, P, assert_within, attention, cache_struct, frequencies, gm, half_step, m, make_cache, rotate)

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2M1 = "e2m1"


# ------------------------------------------------------------------ definitions in 64 bits

def nearest_even(x, values):
    """Index of the nearest of ascending values (1-D), of two equally near ones the even index."""
    values = values.to(x.device)
    hi = torch.bucketize(x, values).clamp(1, len(values) - 1)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    return torch.where((b < a) | ((a == b) & (hi % 2 == 0)), hi, lo)


def e4m3_values():
    return torch.arange(127, dtype=torch.uint8).view(E4M3).double()


def quantize(x, scale):
    """x [..., d] in 64 bits, scale (broadcast over all but d): (codes without and with sign [..., d], scale bytes)."""
    blocks = x.unflatten(-1, (-1, 16))
    g = scale.double().abs()[..., None, None] if torch.is_tensor(scale) else abs(scale)
    sbytes = nearest_even(blocks.abs().amax(-1, keepdim=True) / (6 * g), e4m3_values())
    s = e4m3_values().to(x.device)[sbytes]
    q = torch.where(s > 0, blocks.abs() / torch.where(s > 0, s * g, torch.ones_like(s)), torch.zeros_like(blocks))
    return nearest_even(q, VALUES).flatten(-2), sbytes.squeeze(-1)


def unpack(rows, d, scale=None):
    """Rows of a 4-bit cache [..., d/2 + d/16] as 64-bit values."""
    c = torch.stack((rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4), -1).flatten(-2).long()
    x = VALUES.to(rows.device)[c % 8] * (1 - 2 * (c // 8))
    s = rows[..., d // 2:].contiguous().view(E4M3).double()
    x = (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)
    return x if scale is None else x * scale.double()


def random_rows(shape, d, gen):
    """Random rows: codes of any kind, scales around one."""
    rows = torch.randint(0, 256, shape + (d // 2 + d // 16,), generator=gen, device="cuda", dtype=torch.uint8)
    s = (torch.rand(shape + (d // 16,), generator=gen, device="cuda") + 0.2).to(E4M3)
    rows[..., d // 2:] = s.view(torch.uint8)
    return rows


def make_any(B, Hkv, d, page, max_pages, elem, gen, gap=0):
    """make_cache for all three types; gap in units of 16 bytes for a 4-bit one."""
    if elem != E2M1:
        return make_cache(B, Hkv, d, page, max_pages, elem, gen, gap=gap)
    n, row = B * max_pages + 2, d // 2 + d // 16
    flat = torch.zeros(2, n, Hkv * page * row + 16 * gap, dtype=torch.uint8, device="cuda")
    k, v = (flat[i, :, :Hkv * page * row].view(n, Hkv, page, row) for i in (0, 1))
    for c in (k, v):
        c.copy_(random_rows((n, Hkv, page), d, gen))
    table = torch.randperm(n, generator=gen, device="cuda")[:B * max_pages].to(torch.int32).view(B, max_pages)
    return k, v, table, tuple(torch.rand(Hkv, generator=gen, device="cuda") + 0.5 for _ in (0, 1))


def rows_of(cache, row, n):
    """The first n cached rows of a sequence, [Hkv, n, bytes or elements]."""
    at = torch.arange(n, device=cache.device)
    p = cache.shape[2]
    if cache.dtype is E4M3:
        x = cache.view(torch.uint8)[row[at // p].long(), :, at % p].view(E4M3)
    else:
        x = cache[row[at // p].long(), :, at % p]
    return x.transpose(0, 1)


def states(cache, scale, row, n, d):
    x = rows_of(cache, row, n)
    x = unpack(x, d) if cache.dtype is torch.uint8 else x.double()
    return x if scale is None else x * scale.double()[:, None, None]


# ------------------------------------------------------------------------------- host side

E2 = dict(elem=3, k_scale=P, v_scale=P, page_stride=2 * 16 * 72)


@pytest.mark.parametrize("fault,code", [
    (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(page_size=12), -1), (dict(page_stride=2 * 16 * 72 - 16), -1),
    (dict(page_stride=2 * 16 * 72 + 8), -2), (dict(elem=4), -1), (dict(elem=2), -1), (dict(d=32), -1)])
def test_4_bit_cache_refusals(m, fault, code):
    c = ctypes.byref(cache_struct(m, **dict(E2, **fault)))
    assert m.lib.mercury_kv_append(P, None, P, None, 2, 5, c, P, None, None, None, None, 0, None, None, None) == code
    assert m.lib.mercury_attn_paged(P, None, c, P, None, 2, 4, 1, 1, P, P, None) == code
    assert m.lib.mercury_attn_paged_mass(P, None, c, P, None, 2, 4, 1, 1, P, None, P, 64, None) == code
    assert m.lib.mercury_kv_read(c, P, 2, 64, P, P, None) == code
    assert m.lib.mercury_kv_evict(c, c, P, 64, P, 2, 8, 0, 0, P + 16, P, None, 0, None) == code
    assert m.lib.mercury_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(lens=None), -1), (dict(lse=None), -1), (dict(out=None), -1), (dict(cache=None), -1),
    (dict(width=0), -1), (dict(width=1 << 62), -1), (dict(Hq=3), -1), (dict(Sq=0), -1), (dict(Sq=65), -1), (dict(B=1), -1),
    (dict(q=P + 8), -2), (dict(lse=P + 2), -2), (dict(mass=P + 1), -2), (dict(out=P + 2), -2), (dict(lens=P + 2), -2)])
def test_mass_refusals(m, kw, code):
    a = dict(q=P, cache=ctypes.byref(cache_struct(m)), lens=P, B=2, Hq=4, Sq=1, lse=P, mass=None, out=P, width=64)
    a.update(kw)
    assert m.lib.mercury_attn_paged_mass(a["q"], None, a["cache"], a["lens"], None, a["B"], a["Hq"], a["Sq"], 1, a["lse"],
                                         a["mass"], a["out"], a["width"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(mass=None), -1), (dict(lens=None), -1), (dict(out_lens=None), -1), (dict(kept=None), -1), (dict(cache=None), -1),
    (dict(into=None), -1), (dict(keep=0), -1), (dict(first=-1), -1), (dict(last=-1), -1), (dict(first=5, last=4), -1),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), -1), (dict(keep=65), -1), (dict(width=0), -1), (dict(out_mass=P, out_width=7), -1),
    (dict(out_lens=P), -1), (dict(out_mass=P, out_width=8), -1), (dict(B=3), -1),
    (dict(mass=P + 2), -2), (dict(kept=P + 1), -2), (dict(out_mass=P + 6, out_width=8), -2)])
def test_evict_refusals(m, kw, code):
    a = dict(cache=ctypes.byref(cache_struct(m)), into=ctypes.byref(cache_struct(m)), mass=P, width=64, lens=P, B=2, keep=8,
             first=1, last=2, out_lens=P + 64, kept=P, out_mass=None, out_width=0)
    a.update(kw)
    assert m.lib.mercury_kv_evict(a["cache"], a["into"], a["mass"], a["width"], a["lens"], a["B"], a["keep"], a["first"],
                                  a["last"], a["out_lens"], a["kept"], a["out_mass"], a["out_width"], None) == code


@pytest.mark.parametrize("other", [dict(Hkv=1, page_stride=16 * 128), dict(d=64), dict(elem=1, k_scale=P, v_scale=P)])
def test_evict_refuses_caches_that_differ(m, other):
    a, b = ctypes.byref(cache_struct(m)), ctypes.byref(cache_struct(m, **other))
    assert m.lib.mercury_kv_evict(a, b, P, 64, P, 2, 8, 0, 0, P + 64, P, None, 0, None) == m.MERCURY_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), -1), (dict(lens=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(S=0), -1), (dict(B=3), -1),
    (dict(k=P + 8), -2), (dict(v=P + 2), -2), (dict(lens=P + 1), -2)])
def test_read_refusals(m, kw, code):
    a = dict(cache=ctypes.byref(cache_struct(m)), lens=P, B=2, S=64, k=P, v=P)
    a.update(kw)
    assert m.lib.mercury_kv_read(a["cache"], a["lens"], a["B"], a["S"], a["k"], a["v"], None) == code


def test_rows_are_not_moved_within_the_same_pages(m):
    """The same table and arrays are refused; of the same arrays with another table only what else is wrong."""
    def evict(k=P, v=P, table=P):
        a, b = cache_struct(m), cache_struct(m, k=k, v=v, block_table=table)
        return m.lib.mercury_kv_evict(ctypes.byref(a), ctypes.byref(b), P, 64, P, 2, 8, 0, 0, P + 64, P, None, 0, None)

    for kw in (dict(), dict(k=P + 4096), dict(v=P + 4096)):
        assert evict(**kw) == m.MERCURY_EINVAL and b"own pages" in m.lib.mercury_last_error()
    assert m.lib.mercury_kv_read(ctypes.byref(cache_struct(m)), P, 2, 64, P, P, None) == m.MERCURY_EINVAL
    assert b"two tensors" in m.lib.mercury_last_error()


# ---------------------------------------------------------------------------------- append

@pytest.mark.gpu
@pytest.mark.parametrize("scale", ["random", 1.0])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,S,d,page,rot,interleaved,past,new", [
    (1, 4, 2, 1, 128, 16, 128, False, [0], None),
    (3, 8, 1, 1, 64, 16, 64, True, [15, 16, 47], None),
    (2, 6, 3, 40, 128, 16, 128, False, [0, 5], [40, 17]),
    (3, 2, 2, 21, 64, 8, 32, True, [3, 0, 60], [0, 21, 1]),
    (2, 5, 5, 9, 128, 8, 24, False, [0, 30], None),
    (1, 64, 8, 300, 128, 64, 128, True, [100011], [299]),
    (2, 0, 4, 33, 64, 24, 0, False, [1, 2], None),
    (2, 3, 1, 70, 128, 40, 96, False, [7, 0], None),
    (1, 3, 2, 50, 64, 16, 34, True, [2], None),
])
def test_4_bit_append_stores_the_nearest_codes(gm, scale, aligned, B, Hq, Hkv, S, d, page, rot, interleaved, past, new):
    gen = torch.Generator("cuda").manual_seed(S * 7 + d + rot)
    first_page = min(past) // page  # far positions without a far table's memory
    max_pages = -(-(max(past) + S) // page)
    used = max_pages - first_page
    n = B * used + 2
    k_cache, v_cache = (random_rows((n, Hkv, page), d, gen) for _ in range(2))
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, first_page:] = torch.randperm(n, generator=gen, device="cuda")[:B * used].to(torch.int32).view(B, used)
    ks, vs = (torch.rand(Hkv, generator=gen, device="cuda") + 0.3 if scale == "random" else torch.full((Hkv,), scale, device="cuda")
              for _ in range(2))
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    before = k_cache.clone(), v_cache.clone()
    heads = Hq + 2 * Hkv
    pad = 0 if aligned else 1
    qkv = torch.randn(B, S, heads, d + pad, generator=gen, device="cuda").to(BF16).transpose(1, 2)[..., pad:]
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    past_t = torch.tensor(past, dtype=torch.int32, device="cuda")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    plan = gm.mercury_rope_init(rot, interleaved=interleaved) if rot else None
    kw = {}
    if Hq:
        kw = dict(q=q, q_out=q)  # in place
        q_was = q.clone()
    gm.mercury_kv_append(cache, k, v, past_t, new_lens=new_t, rope=plan, **kw)
    gm.mercury_sync_status()
    freq = frequencies(rot) if rot else np.zeros(0)
    pos = past_t[:, None].long() + torch.arange(S, device="cuda")
    rk = rotate(k, pos, freq, interleaved)
    live = torch.zeros(n, page, dtype=torch.bool, device="cuda")
    for b in range(B):
        c = S if new is None else new[b]
        at = past[b] + torch.arange(c, device="cuda")
        pg, row = table[b][at // page].long(), at % page
        live[pg, row] = True
        for got, ref, sc in ((k_cache, rk[b, :, :c], ks), (v_cache, v[b, :, :c].double(), vs)):
            stored = got[pg, :, row].transpose(0, 1)  # [Hkv, c, bytes]
            codes, sbytes = quantize(ref, sc[:, None])
            mine = torch.stack((stored[..., :d // 2] & 15, stored[..., :d // 2] >> 4), -1).flatten(-2)
            assert torch.equal(stored[..., d // 2:].long(), sbytes)
            assert torch.equal((mine & 7).long(), codes)
            some = codes > 0
            assert torch.equal((mine >> 3)[some].bool(), (ref < 0)[some])
        if Hq:
            rq = rotate(q_was[b:b + 1, :, :c], pos[b:b + 1, :c], freq, interleaved)
            assert_within(q[b:b + 1, :, :c], rq, half_step(rq, BF16) + 1e-5, "queries")
            assert torch.equal(q[b, :, c:], q_was[b, :, c:])
    for got, was in zip((k_cache, v_cache), before):
        assert torch.equal(got.transpose(1, 2)[~live], was.transpose(1, 2)[~live])


@pytest.mark.gpu
@pytest.mark.parametrize("g", [1.0, 0.5, 3.0, 1 / 3, 0.7, -5.0, 1.1e-3, 2.0 ** -40, 2.0 ** 40])
@pytest.mark.parametrize("aligned", [True, False])
def test_4_bit_append_of_every_kind_of_block(gm, g, aligned):
    """Blocks of all magnitudes, with ties, zeros and subnormal scales, against the exact quotients."""
    gen = torch.Generator("cuda").manual_seed(11)
    S, Hkv, d = 512, 2, 128
    x = torch.randn(1, Hkv, S, d, generator=gen, device="cuda")
    # block magnitudes over e4m3's whole range and beyond its ends
    x = x.unflatten(-1, (-1, 16)) * torch.exp2(torch.randint(-14, 13, (1, Hkv, S, 8, 1), generator=gen, device="cuda").float())
    x = x.flatten(-2)
    few = torch.randint(-24, 25, x.shape, generator=gen, device="cuda").float() / 4  # few bits: many ties
    x[:, :, : S // 2] = few[:, :, : S // 2] * torch.exp2(torch.randint(-3, 3, (1, Hkv, S // 2, 1), generator=gen, device="cuda").float())
    x[:, :, :4] = 0
    v = torch.empty(1, Hkv, S, d + 8, dtype=BF16, device="cuda")[..., 8 if aligned else 1:][..., :d]
    v.copy_(x * abs(g))
    k_cache, v_cache = (torch.zeros(S // 16, Hkv, 16, 72, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.arange(S // 16, dtype=torch.int32, device="cuda").view(1, -1)
    sc = torch.full((Hkv,), g, device="cuda")
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=sc, v_scale=sc)
    gm.mercury_kv_append(cache, v, v, torch.zeros(1, dtype=torch.int32, device="cuda"))
    gm.mercury_sync_status()
    codes, sbytes = quantize(v[0].double(), sc[:, None])
    for c in (k_cache, v_cache):
        stored = rows_of(c, table[0], S)
        mine = torch.stack((stored[..., :64] & 15, stored[..., :64] >> 4), -1).flatten(-2)
        assert torch.equal(stored[..., 64:].long(), sbytes)
        assert torch.equal((mine & 7).long(), codes)
        some = codes > 0
        assert torch.equal((mine >> 3)[some].bool(), ((v[0] < 0) != (g < 0))[some])


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [0, 128, 24])
def test_4_bit_append_of_values_that_are_not_finite(gm, rot):
    k = torch.ones(1, 1, 4, 128, dtype=BF16, device="cuda")
    k[0, 0, 0, 40] = math.nan
    k[0, 0, 1, 100] = math.inf
    k[0, 0, 2, 3] = -math.inf
    k[0, 0, 2, 9] = math.nan
    caches = [torch.zeros(1, 1, 8, 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    one = torch.ones(1, device="cuda")
    cache = gm.PagedCache(*caches, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), k_scale=one, v_scale=one)
    plan = gm.mercury_rope_init(rot) if rot else None
    gm.mercury_kv_append(cache, k, k, torch.zeros(1, dtype=torch.int32, device="cuda"), rope=plan)
    gm.mercury_sync_status()
    x = unpack(caches[1][0, 0], 128)  # the values, which are never rotated
    assert torch.isnan(x[0, 32:48]).all() and torch.isfinite(x[0, :32]).all() and torch.isfinite(x[0, 48:]).all()
    assert x[1, 100] == 6 * 448 and torch.isfinite(x[1]).all()
    assert torch.isnan(x[2, :16]).all() and torch.isfinite(x[2, 16:]).all()
    assert (x[3] == 1).all() or (x[3] - 1).abs().max() < 0.07  # (1 / 6 is no e4m3)
    if not rot:
        assert torch.equal(caches[0], caches[1])
    else:
        kx = unpack(caches[0][0, 0], 128)
        assert torch.isfinite(kx[3]).all() and not torch.isfinite(kx[0]).all()


# ------------------------------------------------------------------------------- reading back

@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("B,Hkv,d,page,lens,S", [
    (1, 1, 64, 8, [1], 1), (3, 2, 128, 16, [0, 17, 300], 300), (2, 3, 64, 24, [70, 33], 111), (4, 1, 128, 64, [64, 1, 0, 129], 129)])
def test_read_gives_the_rows_values(gm, elem, B, Hkv, d, page, lens, S):
    gen = torch.Generator("cuda").manual_seed(S)
    k_cache, v_cache, table, (ks, vs) = make_any(B, Hkv, d, page, -(-max(lens) // page) + 1, elem, gen, gap=64)
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (torch.full((B, Hkv, S, d), 9.0, dtype=BF16, device="cuda") for _ in range(2))
    got = gm.mercury_kv_read(cache, lens_t, k_out=k, v_out=v)
    assert got[0] is k and got[1] is v
    got = gm.mercury_kv_read(cache, lens_t, k_out=k, v_out=v)
    assert got[0] is k and got[1] is v
    own_k, own_v = gm.mercury_kv_read(cache, lens_t, S=S)
    gm.mercury_sync_status()
    for b, n in enumerate(lens):
        for got, made, c, s in ((k, own_k, k_cache, ks), (v, own_v, v_cache, vs)):
            ref = states(c, s, table[b], n, d)
            # (the product with the head's scale rounds to 32 bits first)
            assert_within(got[b, :, :n], ref, half_step(ref, BF16) * (1 + 2.0 ** -14), "sequence %d" % b)
            assert (got[b, :, n:] == 9.0).all()
            assert torch.equal(made[b, :, :n], got[b, :, :n]) and (made[b, :, n:] == 0).all()


# ------------------------------------------------------------------------------- attention

def run4(gm, B, Hq, Hkv, Sq, d, page, lens, new=None, causal=True, bf16_out=False, scale=1.0, seed=0, gap=0, spoil=None,
         elem=E2M1):
    gen = torch.Generator("cuda").manual_seed(seed)
    k_cache, v_cache, table, (ks, vs) = make_any(B, Hkv, d, page, max(1, -(-max(lens) // page)) + 1, elem, gen, gap=gap)
    if spoil is not None:
        spoil(k_cache, v_cache, table)
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1
    q = (torch.randn(B, Hq, Sq, d, generator=gen, device="cuda") * scale).to(BF16)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    out = torch.full((B, Hq, Sq, d), 9.0, dtype=BF16 if bf16_out else FP32, device="cuda")
    lse = torch.full((B, Hq, Sq), 9.0, device="cuda")
    call = gm.mercury_attn_paged_bf16 if bf16_out else gm.mercury_attn_paged
    call(q, cache, lens_t, new_lens=new_t, causal=causal, out=out, lse=lse)
    gm.mercury_sync_status()
    return dict(q=q, k=k_cache, v=v_cache, table=table, ks=ks, vs=vs, out=out, lse=lse, cache=cache, lens=lens_t, new=new_t)


def check4(r, lens, new, causal):
    B, Hq, Sq, d = r["q"].shape
    for b in range(B):
        n = Sq if new is None else min(new[b], Sq)
        k, v = states(r["k"], r["ks"], r["table"][b], lens[b], d), states(r["v"], r["vs"], r["table"][b], lens[b], d)
        limits = [lens[b] - n + i + 1 if causal else lens[b] for i in range(n)]
        o, l, eo, el = attention(r["q"][b, :, :n], k, v, limits)
        if r["out"].dtype is BF16:
            eo = eo + half_step(o.abs() + eo, BF16)
        assert_within(r["out"][b, :, :n], o, eo, "O of sequence %d" % b)
        assert_within(r["lse"][b, :, :n], l, el, "LSE of sequence %d" % b)
        assert (r["out"][b, :, n:] == 9.0).all() and (r["lse"][b, :, n:] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bf16_out", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,d,page,lens", [(*s[:5], -(-s[5] // 8) * 8, s[6]) for s in SHAPES])
def test_4_bit_attention_matches_its_formula(gm, bf16_out, B, Hq, Hkv, Sq, d, page, lens):
    r = run4(gm, B, Hq, Hkv, Sq, d, page, lens, bf16_out=bf16_out, seed=sum(lens) + Hq)
    check4(r, lens, None, True)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,d", [(8, 128), (4, 64), (16, 64)])
def test_4_bit_attention_padded_batch(gm, causal, Hq, d):
    lens, new = [500, 3, 40, 2, 0, 130], [4, 3, 0, 5, 2, 1]
    r = run4(gm, 6, Hq, 2, 5, d, 16, lens, new=new, causal=causal, seed=3)
    check4(r, lens, new, causal)


@pytest.mark.gpu
def test_4_bit_attention_large_batches_and_shared_pages(gm):
    gen = np.random.default_rng(5)
    lens = [int(x) for x in gen.integers(0, 200, 500)]
    new = [int(x) for x in gen.integers(0, 2, 500)]
    new[100:420] = [0] * 320
    check4(run4(gm, 500, 2, 1, 1, 64, 16, lens, new=new, seed=6), lens, new, True)

    def share(k, v, table):
        table[1, :3] = table[0, :3]
    check4(run4(gm, 2, 8, 4, 1, 128, 16, [100, 70], gap=8, spoil=share, seed=8), [100, 70], None, True)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (8, 2), (8, 1)])
def test_4_bit_hidden_rows_do_not_matter(gm, d, Hq, Hkv):
    """NaN scales in rows that no row, or only a later row, sees."""
    lens, B, Sq, page = [131, 64, 7, 1300], 4, 4, 16

    def spoil(k, v, table):
        for c in (k, v):
            for b, n in enumerate(lens):
                for at in list(range(n, (n + page - 1) // page * page)) + [n - 1, n - 2]:
                    c[table[b, at // page].long(), :, at % page] = 0x7f

    r = run4(gm, B, Hq, Hkv, Sq, d, page, lens, spoil=spoil, seed=9)
    for b, n in enumerate(lens):
        k, v = states(r["k"], r["ks"], r["table"][b], n - 2, d), states(r["v"], r["vs"], r["table"][b], n - 2, d)
        o, l, eo, el = attention(r["q"][b, :, :2], k, v, [n - 3, n - 2])
        assert_within(r["out"][b, :, :2], o, eo, "O")
        assert_within(r["lse"][b, :, :2], l, el, "LSE")
        assert torch.isnan(r["out"][b, :, 2:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_scale_of_a_value_is_its_16_columns(gm, d):
    lens, page = [300, 40], 16

    def spoil(k, v, table):
        for b, n in enumerate(lens):
            v[table[b, (n - 2) // page].long(), 0, (n - 2) % page, d // 2 + 1] = 0x7f

    r = run4(gm, 2, 4, 1, 3, d, page, lens, spoil=spoil, seed=10)
    clean = r["v"].clone()
    for b, n in enumerate(lens):
        clean[r["table"][b, (n - 2) // page].long(), 0, (n - 2) % page, d // 2 + 1] = 0x38
    bad = torch.isnan(r["out"])
    assert bad[:, :, 1:, 16:32].all() and not bad[:, :, 0].any() and not bad[..., :16].any() and not bad[..., 32:].any()
    out, _ = gm.mercury_attn_paged(r["q"], gm.PagedCache(r["k"], clean, r["table"], k_scale=r["ks"], v_scale=r["vs"]), r["lens"])
    assert torch.equal(out[:, :, 0], r["out"][:, :, 0]) and torch.equal(out[..., 32:], r["out"][..., 32:])


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.7, 1e-3, 30.0])
def test_4_bit_head_scales(gm, scale):
    lens = [700, 33]
    r = run4(gm, 2, 8, 2, 1, 128, 16, lens, seed=12, scale=0.1)
    r["ks"].fill_(scale)
    r["vs"].fill_(scale)
    gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], out=r["out"], lse=r["lse"])
    gm.mercury_sync_status()
    check4(r, lens, None, True)


@pytest.mark.gpu
def test_4_bit_attention_over_a_long_context(gm):
    """64K equal weights: sums neither drift nor truncate."""
    n, d = 65536, 128
    r = run4(gm, 1, 8, 1, 1, d, 64, [n], seed=13)
    r["q"].zero_()
    gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], out=r["out"], lse=r["lse"])
    gm.mercury_sync_status()
    v = states(r["v"], r["vs"], r["table"][0], n, d)
    assert (r["lse"].double() - math.log(n)).abs().max() < 2e-6
    # each of 8 partial sums' roundings is 2^-24 of it, a random walk over n / 32 steps and their joins
    assert (r["out"][0, :, 0].double() - v.mean(1)).abs().max() < 2.0 ** -24 * math.sqrt(n / 32) * v.abs().mean() * 4


# ------------------------------------------------------------------------------------ weights

def weights(r, lse, lens, new, causal, prev, width):
    """(out in 64 bits, its bound), [B,Hkv,width], entries behind a sequence as in prev."""
    B, Hq, Sq, d = r["q"].shape
    Hkv = r["k"].shape[1]
    G = Hq // Hkv
    out, bound = prev.double().clone(), torch.zeros(B, Hkv, width, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = Sq if new is None else min(new[b], Sq)
        k = states(r["k"], r["ks"], r["table"][b], lens[b], d)
        q = r["q"][b, :, :n].double().reshape(Hkv, G, n, d)
        x = torch.einsum("hgnd,hkd->hgnk", q, k) / math.sqrt(d)
        mag = torch.einsum("hgnd,hkd->hgnk", q.abs(), k.abs()) / math.sqrt(d)
        l = lse[b, :, :n].double().reshape(Hkv, G, n, 1)
        at = torch.arange(lens[b], device="cuda")
        lim = torch.tensor([lens[b] - n + i + 1 if causal else lens[b] for i in range(n)], device="cuda")[:, None]
        p = torch.where((at < lim) & torch.isfinite(l), torch.exp(x - l), 0.0)
        l = torch.where(torch.isfinite(l), l, 0.0)
        e = p * (2.0 ** -21 * mag + 2.0 ** -22 * (x.abs() + l.abs()) + 2.0 ** -21)
        add = p.sum((1, 2))
        out[b, :, :lens[b]] += add
        bound[b, :, :lens[b]] = e.sum((1, 2)) + G * n * 2.0 ** -24 * add + 2.0 ** -23 * out[b, :, :lens[b]].abs()
    return out, bound


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("prev", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,d,page,lens,new,causal", [
    (1, 1, 1, 1, 128, 16, [1], None, True),
    (4, 8, 2, 1, 64, 16, [0, 1, 127, 129], None, True),
    (3, 6, 2, 4, 128, 8, [4, 260, 999], None, True),
    (3, 6, 2, 4, 128, 24, [4, 260, 999], None, False),
    (5, 16, 2, 5, 64, 16, [500, 3, 40, 2, 0], [4, 3, 0, 5, 2], True),
    (2, 12, 1, 64, 128, 32, [1000, 64], [64, 33], True),  # 768 rows: three passes of the tensor unit's product
    (3, 16, 1, 4, 64, 16, [500, 4, 130], None, True),     # 64 rows, the most that go by warps
    (3, 13, 1, 5, 64, 16, [500, 5, 1300], None, True),    # 65 rows
    (2, 8, 2, 16, 128, 16, [16, 1100], None, False),      # 64 rows
    (2, 8, 2, 17, 128, 8, [40, 1100], [17, 3], True),     # 68
    (6, 32, 8, 40, 64, 64, [40, 700, 41, 0, 127, 129], None, True),  # 160
    (2, 9, 1, 64, 128, 16, [64, 333], None, True),        # 576
    (40, 3, 3, 1, 128, 16, list(range(40)), None, True),
])
def test_mass_adds_the_weights(gm, elem, prev, B, Hq, Hkv, Sq, d, page, lens, new, causal):
    r = run4(gm, B, Hq, Hkv, Sq, d, page, lens, new=new, causal=causal, seed=sum(lens) + Sq, elem=elem)
    width = max(lens) + 3
    lse = torch.where((r["lse"] == 9.0), math.inf, r["lse"]) if new else r["lse"]
    before = torch.rand(B, Hkv, width, device="cuda") if prev else torch.zeros(B, Hkv, width, device="cuda")
    out = torch.full((B, Hkv, width), 9.0, device="cuda")
    got = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse, new_lens=r["new"], causal=causal,
                                     mass=before if prev else None, out=out)
    gm.mercury_sync_status()
    assert got is out
    ref, bound = weights(r, lse, lens, new, causal, before, width)
    for b, n in enumerate(lens):
        assert_within(out[b, :, :n], ref[b, :, :n], bound[b, :, :n], "sequence %d" % b)
        assert (out[b, :, n:] == 9.0).all()
    mine = before.clone()
    gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse, new_lens=r["new"], causal=causal, mass=mine, out=mine)
    for b, n in enumerate(lens):  # in place, and the same bits
        assert torch.equal(mine[b, :, :n], out[b, :, :n]) and torch.equal(mine[b, :, n:], before[b, :, n:])
    # every row's weights add up to one
    live = sum((Sq if new is None else min(new[b], Sq, )) * (lens[b] > 0) for b in range(B)) * Hq
    if not prev and new is None and min(lens[b] for b in range(B) if lens[b]) >= Sq:
        total = sum(out[b, :, :n].double().sum().item() for b, n in enumerate(lens))
        assert abs(total - live) < 1e-5 * live


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Sq", [12, 13, 16])
def test_mass_over_long_caches(gm, elem, d, Sq):
    """48, 52 and 64 rows over a table of many tiles, where another way is taken."""
    lens, new = [40000, 70, 31111], [Sq, 3, Sq - 1]
    r = run4(gm, 3, 16, 4, Sq, d, 64, lens, new=new, seed=Sq + d, elem=elem)
    lse = torch.where(r["lse"] == 9.0, math.inf, r["lse"])
    got = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse, new_lens=r["new"])
    gm.mercury_sync_status()
    width = got.shape[2]
    ref, bound = weights(r, lse, lens, new, True, torch.zeros(3, 4, width, device="cuda"), width)
    for b, n in enumerate(lens):
        assert_within(got[b, :, :n], ref[b, :, :n], bound[b, :, :n], "sequence %d" % b)
        assert (got[b, :, n:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
def test_mass_of_keys_that_some_rows_see(gm, elem):
    """NaN keys behind the last one count nothing; one that only later rows see is theirs."""
    lens, page = [131, 50], 16

    def spoil(k, v, table):
        for b, n in enumerate(lens):
            for at in list(range(n, (n + page - 1) // page * page)) + [n - 1]:
                if elem is BF16:
                    k[table[b, at // page].long(), :, at % page] = math.nan
                else:
                    k.view(torch.uint8)[table[b, at // page].long(), :, at % page] = 0x7f

    r = run4(gm, 2, 4, 2, 3, 128, page, lens, spoil=spoil, seed=21, elem=elem)
    lse = r["lse"].clone()
    lse[:, :, 2] = math.inf  # the row that sees the NaN: no weight
    out = torch.full((2, 2, 140), 9.0, device="cuda")
    gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse, out=out)
    gm.mercury_sync_status()
    for b, n in enumerate(lens):
        assert torch.isfinite(out[b, :, :n]).all() and (out[b, :, n - 1] == 0).all() and (out[b, :, n:] == 9.0).all()


@pytest.mark.gpu
def test_mass_of_keys_with_infinities(gm):
    """An infinite key's weight is 0 in the rows that it scores -inf in, whatever fills the row tile."""
    r = run4(gm, 1, 3, 1, 1, 128, 16, [100], seed=22, elem=BF16)
    r["q"].copy_(r["q"].abs() + 0.1)
    r["k"][r["table"][0, 2].long(), 0, 5] = -math.inf  # token 37
    out, lse = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    got = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse)
    gm.mercury_sync_status()
    assert torch.isfinite(lse).all() and torch.isfinite(got).all() and got[0, 0, 37] == 0
    assert abs(got.sum().item() - 3) < 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("Sq", [8, 24])
@pytest.mark.parametrize("fill", [math.inf, 1e38, math.nan])
def test_mass_of_rows_that_count_nothing(gm, elem, Sq, fill):
    """A row whose lse is infinite gives nothing, whatever its query holds, and the others what they would."""
    r = run4(gm, 2, 4, 1, Sq, 128, 16, [300, 1100], seed=24, elem=elem)
    lse = r["lse"].clone()
    lse[0, 1, 3] = math.inf
    lse[1, 3, Sq - 1] = -math.inf
    ref, bound = weights(r, lse, [300, 1100], None, True, torch.zeros(2, 1, 1100, device="cuda"), 1100)
    q = r["q"].clone()
    q[0, 1, 3, 5] = q[1, 3, Sq - 1, 64:] = fill
    got = gm.mercury_attn_paged_mass(q, r["cache"], r["lens"], lse)
    gm.mercury_sync_status()
    for b, n in enumerate([300, 1100]):
        assert_within(got[b, :, :n], ref[b, :, :n], bound[b, :, :n], "sequence %d" % b)


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
def test_both_ways_into_the_calls(gm, elem):
    """The short way from Python and the long one (a stream given) make the same call; strided queries too."""
    r = run4(gm, 3, 8, 2, 2, 64, 16, [300, 40, 700], seed=23, elem=elem)
    wide = torch.zeros(3, 2, 8, 96, dtype=BF16, device="cuda").transpose(1, 2)
    q = wide[..., 32:]
    q.copy_(r["q"])
    s = torch.cuda.current_stream()
    outs = [torch.full((3, 2, 700), 9.0, device="cuda") for _ in range(3)]
    gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"], out=outs[0])
    gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"], out=outs[1], stream=s)
    gm.mercury_attn_paged_mass(q, r["cache"], r["lens"], r["lse"], out=outs[2])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    kv = [[torch.full((3, 2, 700, 64), 9.0, dtype=BF16, device="cuda") for _ in range(2)] for _ in range(2)]
    gm.mercury_kv_read(r["cache"], r["lens"], k_out=kv[0][0], v_out=kv[0][1])
    gm.mercury_kv_read(r["cache"], r["lens"], k_out=kv[1][0], v_out=kv[1][1], stream=s)
    assert all(torch.equal(a, b) for a, b in zip(*kv))
    gen = torch.Generator("cuda").manual_seed(7)
    got = []
    for stream in (None, s):
        k2, v2, table2, _ = make_any(3, 2, 64, 16, 8, elem, gen)
        for c in (k2, v2):
            c.view(torch.uint8).zero_()
        table2.copy_(torch.arange(24, device="cuda").view(3, 8))
        into = gm.PagedCache(k2, v2, table2, k_scale=r["ks"], v_scale=r["vs"])
        out_lens, kept = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, 100, dtype=torch.int32, device="cuda")
        gm.mercury_kv_evict(r["cache"], into, outs[0], r["lens"], 100, last=10, out_lens=out_lens, kept=kept, stream=stream)
        got.append((out_lens, kept, k2.view(torch.uint8), v2.view(torch.uint8)))
    gm.mercury_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ----------------------------------------------------------------------------------- eviction

def kept_of(mass, n, keep, first, last):
    """The kept tokens of one head, by the definition."""
    if n <= keep:
        return list(range(n))
    ends = set(range(first)) | set(range(n - last, n))
    key = lambda i: (-math.inf if math.isnan(mass[i]) else mass[i], not math.isnan(mass[i]))  # noqa: E731
    rest = sorted((i for i in range(n) if i not in ends), key=lambda i: (tuple(-x for x in key(i)), i))
    return sorted(ends | set(rest[:keep - first - last]))


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("B,Hkv,d,page,into_page,lens,keep,first,last", [
    (1, 1, 64, 16, 16, [1], 1, 0, 0),
    (3, 2, 128, 16, 16, [0, 40, 300], 64, 4, 16),
    (2, 3, 64, 8, 24, [1025, 1024], 1024, 0, 1),
    (2, 2, 128, 64, 8, [5000, 77], 100, 100, 0),   # the first ones alone
    (2, 1, 64, 24, 16, [2100, 3000], 333, 0, 333),  # the last ones alone
    (1, 5, 128, 16, 32, [9999], 7777, 3, 5),
])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict_keeps_the_heaviest(gm, elem, kind, B, Hkv, d, page, into_page, lens, keep, first, last):
    gen = torch.Generator("cuda").manual_seed(keep + len(lens))
    k, v, table, (ks, vs) = make_any(B, Hkv, d, page, max(1, -(-max(lens) // page)), elem, gen)
    k2, v2, table2, _ = make_any(B, Hkv, d, into_page, -(-keep // into_page), elem, gen)
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1
    width = max(lens) + 2
    mass = torch.exp(3 * torch.randn(B, Hkv, width, generator=gen, device="cuda"))
    if kind == "ties":
        mass = torch.randint(-1, 3, mass.shape, generator=gen, device="cuda").float()
        special = torch.rand(mass.shape, generator=gen, device="cuda")
        mass[special < 0.05] = -0.0
        mass[special > 0.97] = math.nan
        mass[special > 0.98] = math.inf
        mass[special > 0.99] = -math.inf
    cache, into = (gm.PagedCache(a, b, t, k_scale=ks, v_scale=vs) for a, b, t in ((k, v, table), (k2, v2, table2)))
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    was = [x.view(torch.uint8).clone() for x in (k2, v2)]
    out_lens = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    kept = torch.full((B, Hkv, keep), -7, dtype=torch.int32, device="cuda")
    out_mass = torch.full((B, Hkv, keep + 3), 9.0, device="cuda")
    gm.mercury_kv_evict(cache, into, mass, lens_t, keep, first=first, last=last, out_lens=out_lens, kept=kept, out_mass=out_mass)
    gm.mercury_sync_status()
    own_lens, own_kept = gm.mercury_kv_evict(cache, into, mass, lens_t, keep, first=first, last=last)
    gm.mercury_sync_status()
    assert out_lens.tolist() == [min(n, keep) for n in lens] == own_lens.tolist()
    host, slots = mass.cpu(), kept.cpu()
    written = torch.zeros(k2.shape[0], Hkv, into_page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        n2 = min(n, keep)
        at = torch.arange(n2, device="cuda")
        for h in range(Hkv):
            want = kept_of(host[b, h].tolist(), n, keep, first, last)
            assert slots[b, h, :n2].tolist() == want and (slots[b, h, n2:] == -7).all()
            assert own_kept[b, h, :n2].tolist() == want and (own_kept[b, h, n2:] == -1).all()
            src = torch.tensor(want, dtype=torch.long, device="cuda")
            got = out_mass[b, h, :n2]
            assert torch.equal(got.nan_to_num(5.0), mass[b, h, src].nan_to_num(5.0)) and (out_mass[b, h, n2:] == 9.0).all()
            for a, z in ((k, k2), (v, v2)):
                a, z = a.view(torch.uint8), z.view(torch.uint8)
                assert torch.equal(z[table2[b, at // into_page].long(), h, at % into_page], a[table[b, src // page].long(), h, src % page])
            written[table2[b, at // into_page].long(), h, at % into_page] = True
    for z, w in zip((k2, v2), was):
        assert torch.equal(z.view(torch.uint8)[~written], w[~written])


def order_of(mass, n, keep, first, last):
    """kept_of for long sequences, of all heads at once: mass [heads, width] without NaN."""
    at = torch.arange(n, device=mass.device)
    want = torch.where((at < first) | (at >= n - last), math.inf, mass[:, :n].double())
    return torch.sort(want, dim=1, descending=True, stable=True)[1][:, :keep].sort(dim=1)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["spread", "ties"])
@pytest.mark.parametrize("B,Hkv,n,keep", [
    (20, 8, 40000, 3333),   # more heads than SMs, and more tokens than a block holds
    (1, 1, 300000, 70001),  # one head, more tokens than its cluster holds
    (1, 8, 33000, 32999),
    (9, 5, 6000, 16),
])
def test_evict_long_sequences(gm, kind, B, Hkv, n, keep):
    gen = torch.Generator("cuda").manual_seed(n)
    page, d, first, last = 64, 64, 5, 9
    pages = -(-n // page)
    k = random_rows((B * pages, Hkv, page), d, gen)
    table = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32).view(B, pages)
    into_pages = -(-keep // page)
    k2 = torch.zeros(B * into_pages, Hkv, page, 36, dtype=torch.uint8, device="cuda")
    v2 = torch.zeros_like(k2)
    table2 = torch.arange(B * into_pages, dtype=torch.int32, device="cuda").view(B, into_pages)
    one = torch.ones(Hkv, device="cuda")
    cache, into = gm.PagedCache(k, k, table, k_scale=one, v_scale=one), gm.PagedCache(k2, v2, table2, k_scale=one, v_scale=one)
    mass = torch.exp(3 * torch.randn(B, Hkv, n, generator=gen, device="cuda"))
    if kind == "ties":
        mass = torch.randint(0, 4, mass.shape, generator=gen, device="cuda").float()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    small = torch.zeros(B, Hkv, keep, device="cuda")
    got, kept = gm.mercury_kv_evict(cache, into, mass, lens, keep, first=first, last=last, out_mass=small)
    gm.mercury_sync_status()
    assert (got == keep).all()
    want = order_of(mass.view(B * Hkv, n), n, keep, first, last).view(B, Hkv, keep)
    assert torch.equal(kept.long(), want)
    assert torch.equal(small, mass.gather(2, want))
    at = torch.arange(keep, device="cuda")
    for b in {0, B - 1}:
        for h in {0, Hkv - 1}:
            rows = k[table[b, want[b, h] // page].long(), h, want[b, h] % page]
            for z in (k2, v2):
                assert torch.equal(z[table2[b, at // page].long(), h, at % page], rows)


# ------------------------------------------------------------------------------------ together

@pytest.mark.gpu
def test_a_serving_run_with_a_small_cache(gm):
    """Prompt into a 4-bit cache and read back for its attention, decode steps with weights, eviction, more steps."""
    gen = torch.Generator("cuda").manual_seed(31)
    B, Hq, Hkv, d, page, S, keep = 2, 8, 2, 128, 16, 256, 96
    plan = gm.mercury_rope_init(d)

    def new_cache(pages):
        k, v = (torch.zeros(B * pages, Hkv, page, 72, dtype=torch.uint8, device="cuda") for _ in range(2))
        table = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32).view(B, pages)
        return gm.PagedCache(k, v, table, k_scale=torch.ones(Hkv, device="cuda"), v_scale=torch.ones(Hkv, device="cuda"))

    cache = new_cache(20)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(B, h, S, d, generator=gen, device="cuda").to(BF16) for h in (Hq, Hkv, Hkv))
    q = gm.mercury_kv_append(cache, k, v, zero, rope=plan, q=q)
    dense = gm.mercury_kv_read(cache, zero + S, S=S)
    out, lse = gm.mercury_attn_sharded(q, dense[0], dense[1], R=1, shift=0, causal=True)
    # the same rows over the cache itself
    o4, l4 = gm.mercury_attn_paged(q[:, :, -8:].contiguous(), cache, zero + S)
    assert (o4 - out[:, :, -8:]).abs().max() < 2e-2 and (l4 - lse[:, :, -8:]).abs().max() < 1e-2
    mass = gm.mercury_attn_paged_mass(q[:, :, -32:].contiguous(), cache, zero + S, lse[:, :, -32:].contiguous())
    assert abs(mass.sum().item() - B * Hq * 32) < 0.05 * B * Hq * 32
    lens = zero + S
    for step in range(3):
        qs, ks, vs = (torch.randn(B, h, 1, d, generator=gen, device="cuda").to(BF16) for h in (Hq, Hkv, Hkv))
        qs = gm.mercury_kv_append(cache, ks, vs, lens, rope=plan, q=qs)
        lens = lens + 1
        _, l = gm.mercury_attn_paged(qs, cache, lens)
        gm.mercury_attn_paged_mass(qs, cache, lens, l, mass=mass, out=mass)
    into = new_cache(8)
    small = torch.zeros(B, Hkv, 8 * page, device="cuda")
    lens2, kept = gm.mercury_kv_evict(cache, into, mass, lens, keep, first=4, last=32, out_mass=small)
    gm.mercury_sync_status()
    assert lens2.tolist() == [keep, keep]
    # attention over the short cache is attention over the kept tokens
    o, l = gm.mercury_attn_paged(qs, into, lens2)
    for b in range(B):
        kk, vv = (states(c, s, cache.block_table[b], S + 3, d) for c, s in ((cache.k_cache, cache.k_scale), (cache.v_cache, cache.v_scale)))
        at = kept[b].long()[..., None].expand(-1, -1, d)
        ro, rl, eo, el = attention(qs[b], kk.gather(1, at), vv.gather(1, at), [keep])
        assert_within(o[b], ro, eo, "O")
        assert_within(l[b], rl, el, "LSE")
    # and goes on: the next token behind the kept ones, at its own position
    ks, vs = (torch.randn(B, Hkv, 1, d, generator=gen, device="cuda").to(BF16) for _ in range(2))
    gm.mercury_kv_append(into, ks, vs, lens2)
    o2, l2 = gm.mercury_attn_paged(qs, into, lens2 + 1)
    gm.mercury_attn_paged_mass(qs, into, lens2 + 1, l2, mass=small, out=small)
    gm.mercury_sync_status()
    assert (l2 > l).all() and torch.isfinite(o2).all() and (small[:, :, keep] > 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
def test_streams_graphs_and_repetition(gm, elem):
    r = run4(gm, 3, 8, 2, 2, 128, 16, [3000, 40, 700], seed=41, elem=elem)
    gen = torch.Generator("cuda").manual_seed(5)
    k2, v2, table2, _ = make_any(3, 2, 128, 16, 16, elem, gen)
    into = gm.PagedCache(k2, v2, table2, k_scale=r["ks"], v_scale=r["vs"])

    def step(stream=None):
        o, l = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], stream=stream)
        w = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], l, stream=stream)
        n, kept = gm.mercury_kv_evict(r["cache"], into, w, r["lens"], 256, first=4, last=16, stream=stream)
        k, v = gm.mercury_kv_read(into, n, stream=stream)
        return o, l, w, n, kept, k, v

    first = step()
    torch.cuda.synchronize()
    same = lambda x: all(torch.equal(a, b) for a, b in zip(first, x))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert same(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        # (rows that a call leaves as they were hold zeros now)
        assert torch.equal(held[0], first[0]) and torch.equal(held[2], first[2]) and torch.equal(held[3], first[3])
        assert torch.equal(held[4].clamp(min=0), first[4].clamp(min=0)) and torch.equal(held[5], first[5])
    gm.mercury_sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
def test_pages_and_lengths_out_of_range_are_reported(gm, elem):
    r = run4(gm, 3, 4, 2, 1, 128, 16, [100, 60, 90], seed=51, elem=elem)
    keep_out = r["out"].clone()
    gen = torch.Generator("cuda").manual_seed(6)
    k2, v2, table2, _ = make_any(3, 2, 128, 16, 3, elem, gen)
    into = gm.PagedCache(k2, v2, table2, k_scale=r["ks"], v_scale=r["vs"])
    mass = torch.rand(3, 2, 112, device="cuda")

    def calls(lens):
        yield lambda: gm.mercury_attn_paged(r["q"], r["cache"], lens, out=r["out"], lse=r["lse"])
        yield lambda: gm.mercury_attn_paged_mass(r["q"], r["cache"], lens, r["lse"], mass=mass)
        yield lambda: gm.mercury_kv_read(r["cache"], lens)
        yield lambda: gm.mercury_kv_evict(r["cache"], into, mass, lens, 48, first=48)

    def expect(fn):
        fn()
        with pytest.raises(gm.MercuryError) as e:
            gm.mercury_sync_status()
        assert e.value.status == gm.MERCURY_EBOUNDS
        gm.mercury_sync_status()

    good = r["table"].clone()
    for entry in (-1, r["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        r["table"][1, 2] = entry
        for i, fn in enumerate(calls(r["lens"])):
            expect(fn)
            if i == 0:
                assert torch.equal(r["out"][0], keep_out[0]) and torch.equal(r["out"][2], keep_out[2])
                assert torch.isfinite(r["out"]).all()
    r["table"].copy_(good)
    for n in (-3, 10 ** 6, 2 ** 31 - 1):
        for fn in calls(torch.tensor([100, n, 90], dtype=torch.int32, device="cuda")):
            expect(fn)
    into.block_table[2, 1] = 10 ** 6
    expect(lambda: gm.mercury_kv_evict(r["cache"], into, mass, r["lens"], 48, last=48))
    narrow = torch.zeros(3, 2, 64, device="cuda")
    expect(lambda: gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"], mass=narrow))
    expect(lambda: gm.mercury_kv_read(r["cache"], r["lens"], S=64))
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    if elem == E2M1:
        k = torch.ones(3, 2, 2, 128, dtype=BF16, device="cuda")
        for shift in (0, 1):  # both ways of a 4-bit append
            kk = torch.ones(3, 2, 2, 128 + shift, dtype=BF16, device="cuda")[..., shift:]
            for past in ([0, -1, 5], [0, 16 * good.shape[1] - 1, 5], [0, 2 ** 31 - 1, 5], [0, -2 ** 31, 5]):
                cache = gm.PagedCache(r["k"].clone(), r["v"].clone(), good.clamp(min=0), k_scale=r["ks"], v_scale=r["vs"])
                expect(lambda: gm.mercury_kv_append(cache, kk, kk, torch.tensor(past, dtype=torch.int32, device="cuda")))
            expect(lambda: gm.mercury_kv_append(cache, kk, kk, zero, new_lens=torch.tensor([2, 3, -1], dtype=torch.int32, device="cuda")))
        del k


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E2M1])
def test_a_product_whose_end_is_never_told_ends_in_a_timeout(gm, monkeypatch, elem):
    """Weights of many rows: the wait for the tensor unit runs out, the status says so, and the next call is right."""
    r = run4(gm, 2, 8, 2, 32, 128, 16, [300, 200], seed=62, elem=elem)
    first = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"])
    gm.mercury_sync_status()
    monkeypatch.setenv("MERCURY_FAULT", "drop_page_copy")
    monkeypatch.setenv("MERCURY_WAIT_NS", "20000000")
    gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"])
    with pytest.raises(gm.MercuryError) as e:
        gm.mercury_sync_status()
    assert e.value.status == gm.MERCURY_ETIMEOUT
    monkeypatch.delenv("MERCURY_FAULT")
    monkeypatch.delenv("MERCURY_WAIT_NS")
    again = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"])
    gm.mercury_sync_status()
    assert torch.equal(first, again)


@pytest.mark.gpu
def test_a_4_bit_copy_that_never_comes_ends_in_a_timeout(gm, monkeypatch):
    lens = [1700, 20]
    r = run4(gm, 2, 8, 2, 1, 128, 16, lens, seed=61)
    monkeypatch.setenv("MERCURY_FAULT", "drop_page_copy")
    monkeypatch.setenv("MERCURY_WAIT_NS", "20000000")
    gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    with pytest.raises(gm.MercuryError) as e:
        gm.mercury_sync_status()
    assert e.value.status == gm.MERCURY_ETIMEOUT
    monkeypatch.delenv("MERCURY_FAULT")
    monkeypatch.delenv("MERCURY_WAIT_NS")
    out, lse = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    gm.mercury_sync_status()
    assert torch.equal(out, r["out"]) and torch.equal(lse, r["lse"])


@pytest.mark.gpu
def test_binding_refusals_on_the_device(gm):
    r = run4(gm, 2, 4, 2, 1, 128, 16, [20, 9], seed=71)
    q, cache, lens, lse = r["q"], r["cache"], r["lens"], r["lse"]
    mass = torch.zeros(2, 2, 64, device="cuda")
    with pytest.raises(ValueError, match="36 or 72"):
        gm.PagedCache(torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda"), r["table"])
    with pytest.raises(ValueError, match="4-bit cache needs"):
        gm.PagedCache(r["k"], r["v"], r["table"])
    with pytest.raises(gm.MercuryError):  # a page of 12 tokens
        x = torch.zeros(4, 4, 12, 72, dtype=torch.uint8, device="cuda")
        gm.mercury_kv_read(gm.PagedCache(x, x.clone(), r["table"], k_scale=torch.ones(4, device="cuda"), v_scale=torch.ones(4, device="cuda")), lens)
    for kw in (dict(mass=mass[:1]), dict(mass=mass.double()), dict(mass=mass.cpu()), dict(out=mass[..., ::2]), dict(mass=mass, out=mass[:, :, :32].clone()),
               dict(new_lens=lens.long())):
        with pytest.raises((ValueError, TypeError)):
            gm.mercury_attn_paged_mass(q, cache, lens, lse, **kw)
    with pytest.raises((ValueError, TypeError)):
        gm.mercury_attn_paged_mass(q, cache, lens, lse[:, :, 0])
    with pytest.raises(TypeError):
        gm.mercury_kv_evict(cache, None, mass, lens, 8)
    with pytest.raises(gm.MercuryError):
        gm.mercury_kv_evict(cache, cache, mass, lens, 8, first=9)
    for kw in (dict(k_out=torch.zeros(2, 2, 8, 128, device="cuda")), dict(S=8, v_out=torch.zeros(2, 2, 9, 128, dtype=BF16, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            gm.mercury_kv_read(cache, lens, **kw)
    with pytest.raises(TypeError):
        gm.mercury_kv_read(None, lens)


@pytest.mark.gpu
def test_more_refusals_on_the_device(gm):
    r = run4(gm, 2, 4, 2, 1, 128, 16, [20, 9], seed=72)
    cache, lens, mass = r["cache"], r["lens"], torch.zeros(2, 2, 64, device="cuda")
    other = gm.PagedCache(r["k"].clone(), r["v"].clone(), r["table"].clone(), k_scale=r["ks"], v_scale=r["vs"])
    out_lens, kept = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 8, dtype=torch.int32, device="cuda")
    for made in (dict(), dict(out_lens=out_lens, kept=kept)):
        with pytest.raises(gm.MercuryError):  # in place
            gm.mercury_kv_evict(cache, cache, mass, lens, 8, **made)
        for n in (0, 7):
            with pytest.raises(ValueError):
                gm.mercury_kv_evict(cache, other, mass, lens, 8, out_mass=torch.zeros(2, 2, n, device="cuda"), **made)
        for keep in (0, -1):
            with pytest.raises(ValueError):
                gm.mercury_kv_evict(cache, other, mass, lens, keep, **made)
    x = torch.zeros(2, 2, 8, 128, dtype=BF16, device="cuda")
    with pytest.raises(gm.MercuryError):
        gm.mercury_kv_read(cache, lens.clamp(max=8), k_out=x, v_out=x)
    for S in (0, -1):
        with pytest.raises(ValueError):
            gm.mercury_kv_read(cache, lens, S=S)
    gm.mercury_sync_status()
