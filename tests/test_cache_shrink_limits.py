"""The 4-bit cache, weights of cached keys and eviction where they are hardest:
rotated blocks far smaller than what they were turned from, rows of queries far
apart, tokens behind an evicted cache, many rows on the tensor unit.

Bounds as in test_cache_shrink.py.
"""
import numpy as np
import pytest
import torch

from tests.test_cache_shrink import E2M1, make_any, quantize, rows_of, run4, states, weights
from tests.test_paged import (  # noqa: F401
    BF16, E4M3, assert_within, attention, frequencies, gm, half_step, m, rotate, rotation_bound)


# ---------------------------------------------------------------------------------- append

def append4(gm, k, v, past, scale, rope, interleaved, aligned):
    """k, v [B,Hkv,S,d] into a 4-bit cache of pages of 8 that lie in order: the rows of both, [B,Hkv,S,bytes].
    Not aligned: by blocks of 16 elements, element by element."""
    B, Hkv, S, d = k.shape
    pages = -(-(int(past.max()) + S) // 8)
    caches = [torch.zeros(B * pages, Hkv, 8, d // 2 + d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    cache = gm.PagedCache(*caches, table, k_scale=scale, v_scale=scale)
    if not aligned:
        k, v = (torch.nn.functional.pad(x, (1, 0))[..., 1:] for x in (k, v))
    plan = gm.mercury_rope_init(rope[0], base=rope[1], interleaved=interleaved) if rope else None
    gm.mercury_kv_append(cache, k, v, past, rope=plan)
    gm.mercury_sync_status()
    at = past[:, None].long() + torch.arange(S, device="cuda")
    page, b = at // 8, torch.arange(B, device="cuda")[:, None]
    return [c[table[b, page].long(), :, at % 8].transpose(1, 2) for c in caches]


def codes_of(rows, d):
    return torch.stack((rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4), -1).flatten(-2).long()


@pytest.mark.gpu
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("scale", [8 * 4 / 2688, 1e-4, -1e-4, 1e-8])
@pytest.mark.parametrize("d,rot,base,interleaved", [
    (128, 128, 1e4, False), (128, 128, 1e7, False), (64, 64, 5e7, False), (128, 96, 1e6, False), (64, 24, 1e7, False),
    (128, 128, 1e7, True)])
def test_4_bit_append_of_halves_far_apart(gm, aligned, scale, d, rot, base, interleaved):
    """One side of all pairs up to 1e8 times smaller than the other, or zero, at positions where a turn is small: what
    32 bits know of such a block then spans several codes, and several scales."""
    gen = torch.Generator("cuda").manual_seed(rot + int(base) % 97)
    B, Hkv, S = 96, 2, 4
    k = torch.randn(B, Hkv, S, d, generator=gen, device="cuda") * 8
    ratio = torch.logspace(0, 8, B, device="cuda")
    ratio[::8] = torch.inf  # zeros
    small = torch.arange(rot, device="cuda")
    small = small[small % 2 == 0] if interleaved else small[:rot // 2]
    k[..., small] /= ratio[:, None, None, None]
    k[1::2] = k[1::2].roll(rot // 2, -1) if rot == d and not interleaved else k[1::2]  # the other half
    k = k.to(BF16)
    past = (torch.arange(B, device="cuda") % 3).to(torch.int32) * 2  # (position 0 turns nothing)
    sc = torch.full((Hkv,), scale, device="cuda")
    rows = append4(gm, k, k, past, sc, (rot, base), interleaved, aligned)
    pos = past[:, None].long() + torch.arange(S, device="cuda")
    for got, ref in zip(rows, (rotate(k, pos, frequencies(rot, base), interleaved), k.double())):
        codes, sbytes = quantize(ref, sc[:, None])
        mine = codes_of(got, d)
        assert torch.equal(got[..., d // 2:].long(), sbytes)
        assert torch.equal(mine & 7, codes)
        some = codes > 0
        assert torch.equal((mine >> 3)[some].bool(), ((ref < 0) != (scale < 0))[some])


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.01, -0.01, 3.0, -3.0])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 64, True), (128, 24, False), (64, 0, False)])
def test_4_bit_append_gives_the_same_bytes_both_ways(gm, scale, d, rot, interleaved):
    """Zeros of both signs, blocks whose scale is zero, rotated halves that are: a zero's code has no sign, and the bytes
    are the formula's, whichever way they are made."""
    gen = torch.Generator("cuda").manual_seed(rot + d)
    B, Hkv, S = 4, 2, 40
    k = torch.randn(B, Hkv, S, d, generator=gen, device="cuda")
    k *= torch.exp2(torch.randint(-20, 3, (B, Hkv, S, d // 16, 1), generator=gen, device="cuda").float()).expand(-1, -1, -1, -1, 16).flatten(-2)
    k[torch.rand(k.shape, generator=gen, device="cuda") < 0.2] = -0.0
    k[:, :, ::5] = -0.0
    k[:, :, 1::5, :d // 2] = -0.0
    k[:, :, 2::5, d // 2:] = 0.0
    k = k.to(BF16)
    past = torch.tensor([0, 3, 8, 1000], dtype=torch.int32, device="cuda")
    sc = torch.full((Hkv,), scale, device="cuda")
    rope = (rot, 1e4) if rot else None
    rows, other = (append4(gm, k, k, past, sc, rope, interleaved, aligned) for aligned in (True, False))
    pos = past[:, None].long() + torch.arange(S, device="cuda")
    rk = rotate(k, pos, frequencies(rot), interleaved) if rot else k.double()
    for got, same, ref in zip(rows, other, (rk, k.double())):
        assert torch.equal(got, same)
        codes, sbytes = quantize(ref, sc[:, None])
        codes += 8 * ((codes > 0) & ((ref < 0) != (scale < 0)))
        assert torch.equal(got, torch.cat((codes[..., ::2] + 16 * codes[..., 1::2], sbytes), -1).to(torch.uint8))


# ------------------------------------------------------------------------------------ weights

@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("d,Sq,up", [(128, 8, 60), (128, 24, 7), (128, 24, 13), (128, 24, 20), (64, 24, 45), (128, 64, 40), (64, 64, 100)])
def test_mass_does_not_hang_on_other_rows(gm, elem, d, Sq, up):
    """Rows whose queries are 2^up times the others', in elements that all keys are zero in: neither their own weights
    nor the others' lose anything."""
    lens = [300, 1100]

    def spoil(k, v, table):
        k[..., :16 if elem is not E2M1 else 8] = 0  # (codes of zero)

    r = run4(gm, 2, 5, 1, Sq, d, 16, lens, spoil=spoil, seed=25 + up, elem=elem)
    assert (r["q"][..., :16] != 0).any()
    for b, head, i in ((0, 1, 3), (1, 0, 0), (1, 4, Sq - 1)):
        r["q"][b, head, i, 16:] = 0
        r["q"][b, head, i, :16] *= 2.0 ** up
    _, lse = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    got = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse)
    gm.mercury_sync_status()
    assert torch.isfinite(lse).all()
    ref, bound = weights(r, lse, lens, None, True, torch.zeros(2, 1, got.shape[2], device="cuda"), got.shape[2])
    for b, n in enumerate(lens):
        assert_within(got[b, :, :n], ref[b, :, :n], bound[b, :, :n], "sequence %d" % b)


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3])
@pytest.mark.parametrize("heads,Sq", [(2 ** 24 + 64, 1), (2 ** 23 + 40, 3)])
def test_mass_of_more_heads_than_24_bits_count(gm, elem, heads, Sq):
    """The last query heads of many (whose queries overlap in memory), the only ones that count."""
    n, d, last = 40, 64, 30
    r = run4(gm, 1, 1, 1, 1, d, 16, [n], seed=27, elem=elem)
    gen = torch.Generator("cuda").manual_seed(3)
    flat = torch.randn(8 * heads + 64 * Sq, generator=gen, device="cuda").to(BF16)
    q = flat.as_strided((1, heads, Sq, d), (flat.numel(), 8, 64, 1))
    lse = torch.full((1, heads, Sq), torch.inf, device="cuda")
    lse[:, -last:] = 5.0
    out = torch.full((1, 1, n), 9.0, device="cuda")
    gm.mercury_attn_paged_mass(q, r["cache"], r["lens"], lse, out=out)
    gm.mercury_sync_status()
    few = dict(r, q=q[:, -last:])
    ref, bound = weights(few, lse[:, -last:], [n], None, True, torch.zeros(1, 1, n, device="cuda"), n)
    assert_within(out, ref, bound, "weights")


# ----------------------------------------------------------------------------------- eviction

@pytest.mark.gpu
@pytest.mark.parametrize("elem", [E4M3, E2M1])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_eviction_into_a_cache_of_other_scales_is_reported(gm, elem, which):
    """Rows are moved as they are, so other head scales would give them other values; the same ones in tensors of their
    own are fine, and so is a cache of which nothing is kept."""
    r = run4(gm, 2, 4, 2, 1, 128, 16, [0, 90], seed=55, elem=elem)
    gen = torch.Generator("cuda").manual_seed(6)
    k2, v2, table2, _ = make_any(2, 2, 128, 16, 3, elem, gen)
    scales = dict(k_scale=r["ks"].clone(), v_scale=r["vs"].clone())
    into = gm.PagedCache(k2, v2, table2, **scales)
    mass = torch.rand(2, 2, 96, device="cuda")
    lens = r["lens"]
    gm.mercury_kv_evict(r["cache"], into, mass, lens, 48)
    gm.mercury_sync_status()
    scales[which][1] *= 1.0 + 2.0 ** -20
    gm.mercury_kv_evict(r["cache"], into, mass, lens, 48)
    with pytest.raises(gm.MercuryError, match="head scales") as e:
        gm.mercury_sync_status()
    assert e.value.status == gm.MERCURY_EBOUNDS
    gm.mercury_sync_status()
    gm.mercury_kv_evict(r["cache"], into, mass, torch.zeros_like(lens), 48)
    gm.mercury_sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_behind_an_evicted_cache(gm, elem, d):
    """After an eviction a token's place is no longer its position: queries and keys are rotated by mercury_rope at the
    positions that the caller counts on and appended without a plan.  Attention and weights are those over the kept tokens
    and the new ones."""
    gen = torch.Generator("cuda").manual_seed(d)
    B, Hq, Hkv, page, S, keep, more = 2, 6, 2, 16, 200, 64, 5
    plan = gm.mercury_rope_init(d)

    def new_cache(pages):
        k, v, _, scales = make_any(B, Hkv, d, page, pages, elem, gen)
        table = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32).view(B, pages)
        if scales[0] is not None:
            scales = [torch.full((Hkv,), 0.01, device="cuda") for _ in range(2)]
        return gm.PagedCache(k, v, table, k_scale=scales[0], v_scale=scales[1])

    def token(b):
        return [torch.randn(B, h, b, d, generator=gen, device="cuda").to(BF16) for h in (Hq, Hkv, Hkv)]

    cache, into = new_cache(14), new_cache(6)
    lens = torch.tensor([S, 150], dtype=torch.int32, device="cuda")
    q, k, v = token(S)
    q = gm.mercury_kv_append(cache, k, v, torch.zeros_like(lens), new_lens=lens, rope=plan, q=q)
    mass = torch.rand(B, Hkv, S, generator=gen, device="cuda")
    at, kept = gm.mercury_kv_evict(cache, into, mass, lens, keep, first=4, last=16)
    gm.mercury_sync_status()
    assert at.tolist() == [keep, keep]
    short = [torch.stack([states(c, s, into.block_table[b], keep, d) for b in range(B)])
             for c, s in ((into.k_cache, into.k_scale), (into.v_cache, into.v_scale))]
    for c, s, got in ((cache.k_cache, cache.k_scale, short[0]), (cache.v_cache, cache.v_scale, short[1])):
        for b in range(B):  # the tokens that were kept, each rotated at its own position
            rows = states(c, s, cache.block_table[b], int(lens[b]), d)
            assert torch.equal(got[b], rows.gather(1, kept[b].long()[..., None].expand(-1, -1, d)))
    for step in range(more):
        q, k, v = token(1)
        pos = (lens + step)[:, None].contiguous()
        q, rk = (gm.mercury_rope(x, plan, positions=pos) for x in (q, k))
        gm.mercury_kv_append(into, rk, v, at + step)
        out, lse = gm.mercury_attn_paged(q, into, at + step + 1)
        w = gm.mercury_attn_paged_mass(q, into, at + step + 1, lse)
        gm.mercury_sync_status()
        n = keep + step + 1
        ref = rotate(k, pos.long(), frequencies(d), False)
        # rotated in 32 bits (6e-7 of a pair) and rounded to bf16
        assert_within(rk, ref, half_step(ref, BF16) + rotation_bound(k, d // 2, False), "key")
        for x, c, s, got in ((rk, into.k_cache, into.k_scale, short[0]), (v, into.v_cache, into.v_scale, short[1])):
            for b in range(B):
                rows = states(c, s, into.block_table[b], n, d)
                assert torch.equal(rows[:, :keep], got[b])
                if elem is BF16:
                    assert torch.equal(rows[:, n - 1], x[b, :, 0].double())
                elif elem is E2M1:
                    codes, sbytes = quantize(x[b, :, 0].double(), s)
                    new = rows_of(c, into.block_table[b], n)[:, n - 1]
                    assert torch.equal(codes_of(new, d) & 7, codes) and torch.equal(new[:, d // 2:].long(), sbytes)
        r = dict(q=q, k=into.k_cache, ks=into.k_scale, table=into.block_table)
        for b in range(B):
            kk, vv = (states(c, s, into.block_table[b], n, d) for c, s in ((into.k_cache, into.k_scale), (into.v_cache, into.v_scale)))
            o, l, eo, el = attention(q[b], kk, vv, [n])
            assert_within(out[b], o, eo, "O")
            assert_within(lse[b], l, el, "LSE")
        wide = w.shape[2]
        ref, bound = weights(r, lse, [n, n], None, True, torch.zeros(B, Hkv, wide, device="cuda"), wide)
        assert_within(w, ref, bound, "weights")


# ------------------------------------------------- weights of many rows, where few were tested

@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("d,Hq,Sq", [(128, 4, 50), (64, 6, 24), (128, 10, 64), (64, 8, 9)])
def test_mass_of_many_rows_and_keys_that_some_see(gm, elem, d, Hq, Sq):
    """NaN keys behind the last one and infinite or NaN ones that only rows without weight see, with pages whose tail is
    not in the table."""
    lens, page = [131, 500, Sq], 16

    def spoil(k, v, table):
        for b, n in enumerate(lens):
            for at in list(range(n, (n + page - 1) // page * page)) + [n - 1]:
                if elem is BF16:
                    k[table[b, at // page].long(), :, at % page] = float("inf") if at % 2 else float("nan")
                else:
                    k.view(torch.uint8)[table[b, at // page].long(), :, at % page] = 0x7f

    r = run4(gm, 3, Hq, 2, Sq, d, page, lens, spoil=spoil, seed=31, elem=elem)
    lse = r["lse"].clone()
    lse[:, :, Sq - 1] = torch.inf  # the row that sees the bad key
    out = torch.full((3, 2, 512), 9.0, device="cuda")
    gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse, out=out)
    gm.mercury_sync_status()
    clean = r["k"].clone()
    for b, n in enumerate(lens):
        clean.view(torch.uint8)[r["table"][b, (n - 1) // page].long(), :, (n - 1) % page] = 0
    ref, bound = weights(dict(r, k=clean), lse, lens, None, True, torch.zeros(3, 2, 512, device="cuda"), 512)
    for b, n in enumerate(lens):
        assert_within(out[b, :, :n], ref[b, :, :n], bound[b, :, :n], "sequence %d" % b)
        assert (out[b, :, n - 1] == 0).all() and (out[b, :, n:] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [8, 40])
def test_mass_of_many_rows_and_infinite_keys(gm, Sq):
    """An infinite key in a full tile, whose weight is 0 in all rows: they all score -inf."""
    r = run4(gm, 1, 6, 2, Sq, 128, 16, [1000], seed=22, elem=BF16)
    r["q"].copy_(r["q"].abs() + 0.1)
    r["k"][r["table"][0, 20].long(), 1, 5] = -torch.inf  # token 325
    out, lse = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    got = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse)
    gm.mercury_sync_status()
    assert torch.isfinite(lse).all() and torch.isfinite(got).all() and got[0, 1, 325] == 0
    assert (got.sum((0, 2)) - 3 * Sq).abs().max() < 1e-4 * Sq


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [E4M3, E2M1])
@pytest.mark.parametrize("Sq", [1, 12, 30])
@pytest.mark.parametrize("scale", [-0.7, -1e-3, 2.0 ** -40])
def test_mass_with_head_scales_of_any_sign(gm, elem, Sq, scale):
    lens = [700, 33]
    r = run4(gm, 2, 8, 2, Sq, 128, 16, lens, seed=12, scale=0.1, elem=elem)
    r["ks"].fill_(scale)
    _, lse = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    got = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], lse)
    gm.mercury_sync_status()
    wide = got.shape[2]
    ref, bound = weights(r, lse, lens, None, True, torch.zeros(2, 2, wide, device="cuda"), wide)
    assert_within(got, ref, bound, "weights")


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("d", [64, 128])
def test_mass_of_many_rows_with_pages_and_lengths_out_of_range(gm, elem, d):
    lens, Sq = [100, 300, 90], 40
    r = run4(gm, 3, 4, 2, Sq, d, 16, lens, seed=51, elem=elem)
    first = gm.mercury_attn_paged_mass(r["q"], r["cache"], r["lens"], r["lse"])
    gm.mercury_sync_status()
    good = r["table"].clone()

    def expect(lens_t, **kw):
        got = gm.mercury_attn_paged_mass(r["q"], r["cache"], lens_t, r["lse"], **kw)
        with pytest.raises(gm.MercuryError) as e:
            gm.mercury_sync_status()
        assert e.value.status == gm.MERCURY_EBOUNDS
        gm.mercury_sync_status()
        return got

    for entry in (-1, r["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        r["table"][1, 5] = entry  # tokens 80 to 95 count as zeros: exp(-lse) of each row that sees them
        got = expect(r["lens"])
        want = torch.exp(-r["lse"][1].double()).view(2, 2 * Sq).sum(1)
        assert (got[1, :, 80:96] / want[:, None] - 1).abs().max() < 1e-5
        got[1, :, 80:96] = first[1, :, 80:96]
        assert torch.equal(got, first)
    r["table"].copy_(good)
    for n in (-3, 10 ** 6, 2 ** 31 - 1):
        got = expect(torch.tensor([100, n, 90], dtype=torch.int32, device="cuda"))
        assert torch.equal(got[0], first[0]) and torch.equal(got[2], first[2])
    narrow = expect(r["lens"], mass=torch.zeros(3, 2, 256, device="cuda"))
    assert torch.equal(narrow[0, :, :100], first[0, :, :100])
    expect(r["lens"], new_lens=torch.tensor([Sq, Sq + 1, -1], dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("elem", [BF16, E4M3, E2M1])
def test_mass_of_many_rows_on_streams_and_in_graphs(gm, elem):
    r = run4(gm, 3, 8, 2, 64, 128, 16, [3000, 64, 700], seed=41, elem=elem)  # 256 rows
    other = run4(gm, 1, 3, 1, 30, 128, 16, [900], seed=42, elem=elem)
    calls = [lambda x=x, s=None: gm.mercury_attn_paged_mass(x["q"], x["cache"], x["lens"], x["lse"], stream=s) for x in (r, other)]
    first = [f() for f in calls]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in calls]
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):  # at the same time, both holding the tensor unit's memory
        got = [[f(s=side) for f, side in zip(calls, sides)] for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [f() for f in calls + calls]
    for _ in range(3):
        for x in held:
            x.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, first + first))
    gm.mercury_sync_status()
