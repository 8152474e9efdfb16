"""The 4-bit cache, weights of cached keys and eviction where they are hardest:
rotated blocks far smaller than what they were turned from, rows of queries far
apart.

Bounds as in test_cache_shrink.py.
"""
import numpy as np
import pytest
import torch

from tests.test_cache_shrink import E2M1, make_any, quantize, run4, weights
from tests.test_paged import BF16, E4M3, assert_within, frequencies, gm, m, rotate  # noqa: F401


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
