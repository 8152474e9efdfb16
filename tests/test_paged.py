"""Rotary positions, the paged cache append and attention over a paged cache,
against their definitions in 64 bits.

Bounds.  A rounding is off by at most half a step: 2^-8 of the value for bf16,
2^-24 for fp32, 2^-4 for e4m3 (2^-10 absolutely below its smallest normal
2^-6).  Rotation: the angle's reduction leaves 2^-25 of half a turn and the
32-bit sine and cosine and two products round a few times more: 6e-7 of
|a| + |b| covers them.  Attention: a score is a sum of d products in a 32-bit
accumulator (2^-21 of the sum of their magnitudes, over sqrt(d), allows for
its truncation), P is kept to 2^-17 or better and an accumulator that takes the keys in
steps of 16 to 128 loses 2^-23 a step; each is relative to sum p |v|.
"""
import concurrent.futures
import ctypes
import math
import sys

import numpy as np
import pytest
import torch

from tests.conftest import ROOT  # noqa: F401  (puts the repository on the path)

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def m():
    from long_context_sharded_gb300 import build
    build.build()
    from long_context_sharded_gb300 import mercury
    return mercury


@pytest.fixture(scope="module")
def gm(m):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


# ------------------------------------------------------------------ definitions in 64 bits

def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, fast=32.0, slow=1.0):
    i = np.arange(rot // 2)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = 1.0 / base ** (2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        f = f / factor * (1 - g) + f * g
    return f


def rotate(x, pos, freq, interleaved, magnitude=1.0, inverse=False):
    """x [B,H,S,d] (any device), pos [B,S] -> 64-bit rotated copy."""
    y = x.double().clone()
    n = len(freq)
    first = torch.arange(n) * 2 if interleaved else torch.arange(n)
    second = first + (1 if interleaved else n)
    t = pos.double()[:, None, :, None] * torch.tensor(np.asarray(freq), dtype=torch.float64, device=x.device)
    c, s = t.cos() * magnitude, t.sin() * magnitude * (-1 if inverse else 1)
    a, b = x[..., first].double(), x[..., second].double()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def rotation_bound(x, n, interleaved, magnitude=1.0):
    """6e-7 (|a| + |b|) on both elements of a pair."""
    e = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    first = torch.arange(n) * 2 if interleaved else torch.arange(n)
    second = first + (1 if interleaved else n)
    s = 6e-7 * abs(magnitude) * (x[..., first].double().abs() + x[..., second].double().abs())
    e[..., first], e[..., second] = s, s
    return e


def half_step(ref, dtype):
    """Bound of one rounding of ref to dtype."""
    if dtype is E4M3:
        return torch.clamp(ref.abs() * 2.0 ** -4, min=2.0 ** -10)
    return ref.abs() * (torch.finfo(dtype).eps / 2)


def gather_states(cache, scale, row, n):
    """The first n states of a sequence [Hkv, n, d] in 64 bits."""
    P = cache.shape[2]
    at = torch.arange(n, device=cache.device)
    x = cache.view(torch.uint8)[row[at // P].long(), :, at % P].view(cache.dtype) if cache.dtype is E4M3 \
        else cache[row[at // P].long(), :, at % P]
    x = x.double().transpose(0, 1)
    return x if scale is None else x * scale.double()[:, None, None]


def attention(q, k, v, limits):
    """q [Hq,Sq,d], k/v [Hkv,n,d] 64 bit, limits[i] keys seen by token i: O, LSE and their bounds."""
    Hq, Sq, d = q.shape
    G = Hq // k.shape[0]
    o = torch.zeros(Hq, Sq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((Hq, Sq), -math.inf, dtype=torch.float64, device=q.device)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    for i in range(Sq):
        n = min(max(limits[i], 0), k.shape[1])
        if n == 0:
            continue
        qi = q[:, i].double().reshape(-1, G, d)
        x = qi @ k[:, :n].transpose(1, 2) / math.sqrt(d)
        ds = 2.0 ** -21 * (qi.abs() @ k[:, :n].abs().transpose(1, 2) / math.sqrt(d)).amax(-1).reshape(Hq)
        p = torch.softmax(x, -1)
        o[:, i] = (p @ v[:, :n]).reshape(Hq, d)
        lse[:, i] = torch.logsumexp(x, -1).reshape(Hq)
        spread = (p @ v[:, :n].abs()).reshape(Hq, d)
        eo[:, i] = (2 * ds + 2.0 ** -17 + (n / 128 + 40) * 2.0 ** -23)[:, None] * spread
        el[:, i] = ds + (n / 128 + 40) * 2.0 ** -23 + 2.0 ** -22 * lse[:, i].abs()
    return o, lse, eo, el


def assert_within(got, ref, bound, what):
    got, ref, bound = got.double(), ref.double(), bound.double()
    assert got.shape == ref.shape, what
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)), what + ": finite in other places"
    assert torch.equal(ref[~fin], got[~fin]), what
    over = (got - ref).abs()[fin] - bound[fin]
    assert over.numel() == 0 or over.max() <= 0, "%s: %.3g beyond its bound" % (what, over.max().item())


# ------------------------------------------------------------------------------- host side

@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0)),
    ("yarn", dict(factor=16.0, original_length=4096)),
    ("yarn", dict(factor=2.0, original_length=100, beta_fast=8.0, beta_slow=0.5))])
@pytest.mark.parametrize("rot", [4, 24, 64, 128, 256])
def test_frequencies_follow_their_formulas(m, scaling, kw, rot):
    f, mag = m.mercury_rope_frequencies(rot, 500000.0, scaling, **kw)
    ref = frequencies(rot, 500000.0, scaling, kw.get("factor", 1.0), kw.get("original_length", 0.0),
                      kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    np.testing.assert_allclose(f, ref, rtol=1e-13)
    assert mag == pytest.approx(0.1 * math.log(kw["factor"]) + 1 if scaling == "yarn" else 1.0, abs=1e-15)


def test_plan_holds_turns_to_their_rounding(m):
    """turns / 2^64 of a turn per position, also after a product with a far
    position modulo one turn."""
    from fractions import Fraction
    f = [1.0, 0.1, 1e-7, 0.0, 6.0, 2 * math.pi, 7.5, 1e5]
    p = m.mercury_rope_init(16, freq=f)
    # pi to 40 digits, so that the exact angle is known to far more than the plan keeps
    two_pi = 2 * Fraction("3.141592653589793238462643383279502884197")
    for i, x in enumerate(f):
        exact = Fraction(x) / two_pi
        for pos in (1, 3, 131071, 2 ** 31 - 1, -5):
            got = Fraction(p.turns[i] * pos % 2 ** 64, 2 ** 64)
            off = (got - exact * pos) % 1
            off = min(off, 1 - off)
            # the quotient by 2 pi rounds once and the 64-bit constant once
            assert off <= abs(pos) * (2 * exact * Fraction(1, 2 ** 53) + Fraction(1, 2 ** 64)), (x, pos)
    assert list(p.turns[8:]) == [0] * 120 and p.rot_dim == 16 and p.interleaved == 0 and p.magnitude == 1.0


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=math.nan),
    dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=64, scaling="linear", factor=math.inf),
    dict(rot_dim=2, scaling="ntk", factor=2.0), dict(rot_dim=64, scaling="yarn", factor=2.0),
    dict(rot_dim=64, scaling="yarn", factor=2.0, original_length=8, beta_fast=1.0, beta_slow=1.0),
    dict(rot_dim=4, freq=[1.0, -0.5]), dict(rot_dim=4, freq=[1.0, math.nan]), dict(rot_dim=4, freq=[1.0, 2.0 ** 21]),
    dict(rot_dim=4, freq=[1.0, 0.5], magnitude=math.inf)])
def test_plan_refusals(m, kw):
    with pytest.raises(m.MercuryError) as e:
        m.mercury_rope_init(**kw)
    assert e.value.status == m.MERCURY_EINVAL


def test_plan_refusals_of_the_binding(m):
    with pytest.raises(ValueError, match="scaling"):
        m.mercury_rope_init(64, scaling="dynamic")
    with pytest.raises(ValueError, match="freq"):
        m.mercury_rope_init(64, freq=[1.0])


P = 0x100000  # fake, 16-byte aligned "device" address: validation never dereferences


def cache_struct(m, **kw):
    f = dict(k=P, v=P, k_scale=None, v_scale=None, block_table=P, page_stride=2 * 16 * 128, table_stride=4, elem=0,
             Hkv=2, d=128, page_size=16, num_pages=8, max_pages=4, B=2)
    f.update(kw)
    return m.PagedCacheStruct(**f)


CACHE_FAULTS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(block_table=None), -1), (dict(elem=2), -1), (dict(elem=1), -1),
    (dict(elem=1, k_scale=P), -1), (dict(d=96), -1), (dict(Hkv=0), -1), (dict(page_size=0), -1),
    (dict(num_pages=0), -1), (dict(max_pages=0), -1), (dict(B=3), -1), (dict(page_stride=2 * 16 * 128 - 8), -1),
    (dict(table_stride=3), -1), (dict(max_pages=1 << 27, table_stride=1 << 27), -1), (dict(Hkv=1 << 20), -1),
    (dict(page_stride=1 << 60, num_pages=1 << 20), -1),
    (dict(k=P + 8), -2), (dict(v=P + 2), -2), (dict(page_stride=2 * 16 * 128 + 4), -2), (dict(block_table=P + 2), -2),
]


@pytest.mark.parametrize("fault,code", CACHE_FAULTS)
def test_cache_refusals(m, fault, code):
    c = ctypes.byref(cache_struct(m, **fault))
    assert m.lib.mercury_kv_append(P, None, P, None, 2, 5, c, P, None, None, None, None, 0, None, None, None) == code
    assert m.lib.mercury_attn_paged(P, None, c, P, None, 2, 4, 1, 1, P, P, None) == code
    assert m.lib.mercury_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(past=None), -1), (dict(cache=None), -1), (dict(S=0), -1),
    (dict(S=1 << 31 >> 1), -1), (dict(q=P), -1), (dict(q=P, q_out=P), -1), (dict(q=P, q_out=P, Hq=40000), -1),
    (dict(k_strides=(-1, 0, 0)), -1), (dict(q=P, q_out=P, Hq=4, q_out_strides=(0, 640, 128)), -1),
    (dict(q=P, q_out=P, Hq=4, q_out_strides=(4 * 640, 128, 128)), -1),
    (dict(k=P + 1), -2), (dict(past=P + 2), -2), (dict(new=P + 2), -2), (dict(q=P, q_out=P + 1, Hq=4), -2)])
def test_append_refusals(m, kw, code):
    a = dict(k=P, v=P, past=P, new=None, S=5, q=None, q_out=None, Hq=0, k_strides=None, q_out_strides=None,
             cache=ctypes.byref(cache_struct(m)))
    a.update(kw)
    st = lambda s: None if s is None else (ctypes.c_longlong * 3)(*s)  # noqa: E731
    assert m.lib.mercury_kv_append(a["k"], st(a["k_strides"]), a["v"], None, 2, a["S"], a["cache"], a["past"], a["new"],
                                   None, a["q"], None, a["Hq"], a["q_out"], st(a["q_out_strides"]), None) == code


def test_append_refuses_a_plan_wider_than_the_head(m):
    plan = m.mercury_rope_init(128)
    c = cache_struct(m, d=64, page_stride=2 * 16 * 64)
    assert m.lib.mercury_kv_append(P, None, P, None, 2, 5, ctypes.byref(c), P, None, ctypes.byref(plan), None, None, 0,
                                   None, None, None) == m.MERCURY_EINVAL
    plan.rot_dim = 7
    assert m.lib.mercury_kv_append(P, None, P, None, 2, 5, ctypes.byref(c), P, None, ctypes.byref(plan), None, None, 0,
                                   None, None, None) == m.MERCURY_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(lens=None), -1), (dict(out=None), -1), (dict(lse=None), -1), (dict(Hq=3), -1),
    (dict(Hq=0), -1), (dict(Sq=0), -1), (dict(Sq=65), -1), (dict(B=1), -1), (dict(strides=(-8, 8, 8)), -1),
    (dict(q=P + 8), -2), (dict(out=P + 8), -2), (dict(lse=P + 2), -2), (dict(lens=P + 1), -2),
    (dict(strides=(512, 132, 128)), -2)])
def test_attention_refusals(m, kw, code):
    a = dict(q=P, lens=P, out=P, lse=P, Hq=4, Sq=1, B=2, strides=None)
    a.update(kw)
    st = None if a["strides"] is None else (ctypes.c_longlong * 3)(*a["strides"])
    for fn in (m.lib.mercury_attn_paged, m.lib.mercury_attn_paged_bf16):
        assert fn(a["q"], st, ctypes.byref(cache_struct(m)), a["lens"], None, a["B"], a["Hq"], a["Sq"], 1, a["out"],
                  a["lse"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(plan=None), -1), (dict(B=0), -1), (dict(H=0), -1), (dict(S=0), -1),
    (dict(H=70000), -1), (dict(B=1 << 16, S=1 << 16), -1), (dict(elem=1), -1), (dict(d=513), -1), (dict(d=32), -1),
    (dict(out_strides=(0, 640, 64)), -1), (dict(out_strides=(1280, 640, 32)), -1), (dict(pos_stride=-1), -1),
    (dict(x=P + 1), -2), (dict(out=P + 1), -2), (dict(pos=P + 2), -2), (dict(elem=2, x=P + 2), -2)])
def test_rope_refusals(m, kw, code):
    plan = m.mercury_rope_init(64)
    a = dict(x=P, out=P, plan=ctypes.byref(plan), pos=None, pos_stride=0, B=2, H=2, S=10, d=64, elem=0,
             out_strides=None)
    a.update(kw)
    st = None if a["out_strides"] is None else (ctypes.c_longlong * 3)(*a["out_strides"])
    assert m.lib.mercury_rope(a["x"], None, a["pos"], a["pos_stride"], 0, a["B"], a["H"], a["S"], a["d"], a["elem"],
                              a["plan"], 0, a["out"], st, None) == code


def test_binding_refuses_cpu_tensors(m):
    plan = m.mercury_rope_init(64)
    x = torch.zeros(1, 2, 3, 64, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA"):
        m.mercury_rope(x, plan)
    with pytest.raises(TypeError, match="bfloat16"):
        m.mercury_rope(x.half(), plan)
    with pytest.raises(ValueError, match="4-D"):
        m.mercury_rope(x[0], plan)
    with pytest.raises(TypeError, match="RopePlan"):
        m.mercury_rope(x, None)
    c = torch.zeros(2, 2, 16, 64, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA"):
        m.PagedCache(c, c, torch.zeros(1, 2, dtype=torch.int32))


# ------------------------------------------------------------------------------------ rope

def test_extension_leaves_what_it_cannot_take(m):
    """The C side of the binding calls nothing for arguments that are not as a call wants them: it returns None,
    leaves no exception, and keeps no reference."""
    m._names()
    plan = ctypes.addressof(m.mercury_rope_init(64))
    struct = cache_struct(m)
    cache = ctypes.addressof(struct)
    x = torch.zeros(1, 2, 3, 64, dtype=BF16)
    lens = torch.zeros(struct.B, dtype=torch.int32)

    class Odd:
        dtype, shape = BF16, (1, 2, 3, 64)

        def get_device(self):
            raise RuntimeError("no")

    for bad in (x, x.float(), x[0], None, 3, "x", Odd(), torch.zeros(0, dtype=BF16)):
        before = sys.getrefcount(bad)
        assert m._fast.rope(bad, plan, None, 0, False, bad) is None
        assert m._fast.rope(bad, plan, bad, 2 ** 70, False, x) is None
        assert m._fast.append(cache, 0, bad, bad, lens, None, plan, bad, bad) is None
        assert m._fast.append(cache, 0, bad, bad, bad, bad, 0, None, None) is None
        assert m._fast.attn(False, bad, cache, 0, lens, None, True, bad, bad) is None
        assert m._fast.attn(True, bad, cache, -1, lens, bad, True, bad, bad) is None
        assert sys.getrefcount(bad) == before
    assert m._fast.rope() is None and m._fast.append(cache) is None and m._fast.attn() is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,S,d,rot", [
    (1, 1, 1, 64, 64), (2, 40, 1, 128, 128), (1, 3, 257, 128, 128), (3, 5, 33, 64, 32), (1, 17, 100, 128, 24),
    (2, 2, 7, 80, 80), (1, 2, 5, 30, 10), (1, 4, 3, 512, 256), (1, 2, 9, 256, 2), (2, 9, 2100, 64, 64)])
def test_rope_matches_its_formula(gm, dtype, interleaved, B, H, S, d, rot):
    gen = torch.Generator("cuda").manual_seed(B * 1000 + S)
    x = torch.randn(B, H, S, d, generator=gen, device="cuda").to(dtype)
    pos = torch.randint(0, 200000, (B, S), generator=gen, device="cuda").to(torch.int32)
    plan = gm.mercury_rope_init(rot, base=500000.0, interleaved=interleaved, scaling="yarn", factor=4.0,
                                original_length=8192)
    mag = 0.1 * math.log(4.0) + 1
    out = gm.mercury_rope(x, plan, pos)
    ref = rotate(x, pos, frequencies(rot, 500000.0, "yarn", 4.0, 8192), interleaved, mag)
    bound = rotation_bound(x, rot // 2, interleaved, mag)
    assert_within(out, ref, bound + half_step(ref.abs() + bound, dtype), "rope")
    assert torch.equal(out[..., rot:], x[..., rot:])
    # in place, and by a start instead of positions
    y = x.clone()
    assert gm.mercury_rope(y, plan, pos, out=y) is y and torch.equal(y, out)
    a = gm.mercury_rope(x, plan, start=77)
    b = gm.mercury_rope(x, plan, torch.arange(77, 77 + S, device="cuda", dtype=torch.int32))
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_and_negative_positions(gm, interleaved):
    """Angles stay exact where 32 bits have no fraction of a turn left."""
    x = torch.randn(1, 2, 6, 128, device="cuda")
    pos = torch.tensor([[0, 2 ** 20 + 1, 10 ** 7 + 3, 2 ** 31 - 1, -1, -2 ** 31]], device="cuda", dtype=torch.int32)
    out = gm.mercury_rope(x, gm.mercury_rope_init(128, interleaved=interleaved), pos)
    ref = rotate(x, pos, frequencies(128), interleaved)
    # the reference's own angle is a 64-bit product: 2^-53 of up to 2^31 radians, and the frequency's rounding again
    bound = rotation_bound(x, 64, interleaved) * (1 + 2.0 ** 31 * 2.0 ** -52 / 6e-7)
    assert_within(out, ref, bound, "far positions")
    assert torch.equal(out[:, :, 0], x[:, :, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 48, 20])
def test_rope_strides(gm, interleaved, rot):
    """Slices of a fused projection, a broadcast input, unaligned rows and a strided output."""
    plan = gm.mercury_rope_init(rot, interleaved=interleaved)
    qkv = torch.randn(2, 19, 7, 128, device="cuda").to(BF16)
    x = qkv.transpose(1, 2)[:, 1:5]  # [B, 4, S, d], heads of the middle
    ref = gm.mercury_rope(x.contiguous(), plan)
    assert torch.equal(gm.mercury_rope(x, plan), ref)
    wide = qkv.clone()
    gm.mercury_rope(x, plan, out=wide.transpose(1, 2)[:, 1:5])
    assert torch.equal(wide.transpose(1, 2)[:, 1:5], ref)
    assert torch.equal(wide[:, :, 0], qkv[:, :, 0]) and torch.equal(wide[:, :, 5:], qkv[:, :, 5:])
    inside = qkv.clone()
    part = inside.transpose(1, 2)[:, 1:5]
    gm.mercury_rope(part, plan, out=part)
    assert torch.equal(inside, wide)
    one = torch.randn(2, 1, 19, 128, device="cuda").to(BF16).expand(2, 4, 19, 128)
    assert torch.equal(gm.mercury_rope(one, plan), gm.mercury_rope(one.contiguous(), plan))
    odd = torch.randn(2 * 4 * 19 * 129 + 1, device="cuda").to(BF16)[1:].view(2, 4, 19, 129)[..., :128]
    assert torch.equal(gm.mercury_rope(odd, plan), gm.mercury_rope(odd.contiguous(), plan))


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(64, 64), (20, 64)])
def test_rope_inverse_is_the_gradient(gm, interleaved, rot, d):
    """inverse=True against the formula's derivative (autograd in 64 bits) and against differences."""
    x = torch.randn(2, 3, 5, d, device="cuda")
    w = torch.randn(2, 3, 5, d, device="cuda")
    pos = torch.randint(0, 5000, (2, 5), device="cuda").to(torch.int32)
    freq = frequencies(rot)
    plan = gm.mercury_rope_init(rot, interleaved=interleaved, magnitude=1.25)
    got = gm.mercury_rope(w, plan, pos, inverse=True)
    x64 = x.double().requires_grad_(True)
    (rotate(x64, pos, freq, interleaved, 1.25) * w.double()).sum().backward()
    bound = rotation_bound(w, rot // 2, interleaved, 1.25) + half_step(x64.grad, FP32)
    assert_within(got, x64.grad, bound, "gradient")
    # a difference along a direction: the map is linear, so any step is exact up to rounding
    u = torch.randn(2, 3, 5, d, device="cuda")
    a = (gm.mercury_rope(x + u, plan, pos).double() * w.double()).sum()
    b = (gm.mercury_rope(x, plan, pos).double() * w.double()).sum()
    slope = (got.double() * u.double()).sum()
    scale = (w.abs().double() * (x.abs() + u.abs()).double().sum(-1, keepdim=True)).sum()
    assert (a - b - slope).abs() <= 4e-6 * scale
    assert torch.equal(w, w)


# ---------------------------------------------------------------------------------- append

def make_cache(B, Hkv, d, page, max_pages, dtype, gen, spare=2, gap=0):
    """Caches of random content, a table of pages in no order and, for e4m3, scales."""
    n = B * max_pages + spare
    whole = torch.randn(2, n, Hkv * page * d + gap, generator=gen, device="cuda")
    if dtype is E4M3:
        whole = (whole * 40).clamp(-448, 448)
    whole = whole.to(dtype)
    k, v = (whole[i, :, :Hkv * page * d].view(n, Hkv, page, d) for i in (0, 1))
    table = torch.randperm(n, generator=gen, device="cuda")[:B * max_pages].to(torch.int32).view(B, max_pages)
    scales = (None, None)
    if dtype is E4M3:
        scales = tuple(torch.rand(Hkv, generator=gen, device="cuda") * 0.02 + 0.01 for _ in (0, 1))
    return k, v, table, scales


def bits(x):
    return x.contiguous().view(torch.uint8 if x.dtype is E4M3 else torch.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,Hq,Hkv,S,d,page,rot,interleaved,past,new", [
    (1, 4, 2, 1, 128, 16, 128, False, [0], None),
    (3, 8, 1, 1, 64, 16, 64, True, [15, 16, 47], None),
    (2, 6, 3, 40, 128, 16, 128, False, [0, 5], [40, 17]),
    (3, 2, 2, 21, 64, 7, 32, True, [3, 0, 60], [0, 21, 1]),
    (2, 5, 5, 9, 128, 1, 24, False, [0, 30], None),
    (1, 64, 8, 300, 128, 64, 128, True, [11], [299]),
    (2, 0, 4, 33, 64, 24, 0, False, [1, 2], None),
])
def test_append_writes_its_rows_and_no_other(gm, dtype, B, Hq, Hkv, S, d, page, rot, interleaved, past, new):
    gen = torch.Generator("cuda").manual_seed(S * 7 + d)
    most = max(past) + S
    k_cache, v_cache, table, (ks, vs) = make_cache(B, Hkv, d, page, -(-most // page), dtype, gen, gap=64)
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    before = k_cache.clone(), v_cache.clone()
    heads = Hq + 2 * Hkv
    qkv = torch.randn(B, S, heads, d, generator=gen, device="cuda").to(BF16).transpose(1, 2)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    past_t = torch.tensor(past, dtype=torch.int32, device="cuda")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    plan = gm.mercury_rope_init(rot, interleaved=interleaved) if rot else None
    kw = {}
    if Hq:
        q_out = torch.full((B, Hq, S, d), 7.0, dtype=BF16, device="cuda")
        kw = dict(q=q, q_out=q_out)
    got = gm.mercury_kv_append(cache, k, v, past_t, new_lens=new_t, rope=plan, **kw)
    gm.mercury_sync_status()
    assert got is kw.get("q_out")
    freq = frequencies(rot) if rot else np.zeros(0)
    pos = past_t[:, None].long() + torch.arange(S, device="cuda")
    rk = rotate(k, pos, freq, interleaved)
    ek = rotation_bound(k, rot // 2, interleaved)
    live = torch.zeros(k_cache.shape[0], page, dtype=torch.bool, device="cuda")
    for b in range(B):
        n = S if new is None else new[b]
        at = past[b] + torch.arange(n, device="cuda")
        pg, row = table[b][at // page].long(), at % page
        live[pg, row] = True
        for c, ref, err, sc in ((k_cache, rk[b, :, :n], ek[b, :, :n], ks), (v_cache, v[b, :, :n].double(), 0 * ek[b, :, :n], vs)):
            stored = c.view(torch.uint8)[pg, :, row].view(c.dtype) if dtype is E4M3 else c[pg, :, row]
            stored = stored.transpose(0, 1).double()
            if dtype is E4M3:
                s64 = sc.double()[:, None, None]
                # the quotient rounds to 32 bits before the byte
                err = err / s64 + (ref / s64).abs() * 2.0 ** -23
                ref = (ref / s64).clamp(-448, 448)
            assert_within(stored, ref, err + half_step(ref.abs() + err, dtype), "sequence %d" % b)
        if Hq:
            ref = rotate(q[b:b + 1, :, :n], pos[b:b + 1, :n], freq, interleaved)
            e = rotation_bound(q[b:b + 1, :, :n], rot // 2, interleaved)
            assert_within(q_out[b:b + 1, :, :n], ref, e + half_step(ref.abs() + e, BF16), "q")
            assert (q_out[b, :, n:] == 7.0).all()
    for c, old in ((k_cache, before[0]), (v_cache, before[1])):
        keep = ~live[:, None, :, None].expand(c.shape)
        assert torch.equal(bits(c)[keep], bits(old)[keep])
    # the queries in place, within the projection
    if Hq:
        whole = qkv.clone(memory_format=torch.preserve_format)
        inside = whole[:, :Hq]
        assert gm.mercury_kv_append(cache, k, v, past_t, new_lens=new_t, rope=plan, q=inside, q_out=inside) is inside
        for b in range(B):
            n = S if new is None else new[b]
            assert torch.equal(inside[b, :, :n], q_out[b, :, :n]) and torch.equal(inside[b, :, n:], q[b, :, n:])
        assert torch.equal(whole[:, Hq:], qkv[:, Hq:])


@pytest.mark.gpu
def test_append_saturates_and_keeps_nan(gm):
    k_cache, v_cache, table, _ = make_cache(1, 1, 64, 4, 1, E4M3, torch.Generator("cuda").manual_seed(0))
    one = torch.ones(1, device="cuda")
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=one, v_scale=one * 0.5)
    k = torch.zeros(1, 1, 1, 64, dtype=BF16, device="cuda")
    k[..., :6] = torch.tensor([1e5, -1e5, math.inf, -math.inf, math.nan, 300.0], device="cuda").to(BF16)
    gm.mercury_kv_append(cache, k, k, torch.zeros(1, dtype=torch.int32, device="cuda"))
    gm.mercury_sync_status()
    row = k_cache.view(torch.uint8)[table[0, 0].long(), 0, 0].view(E4M3).float()
    assert row[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and math.isnan(row[4]) and row[5] == 288.0 or row[5] == 320.0
    row = v_cache.view(torch.uint8)[table[0, 0].long(), 0, 0].view(E4M3).float()
    assert row[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and math.isnan(row[4]) and row[5] == 448.0


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(8, 64), (24, 64), (24, 128), (40, 64), (64, 128), (2, 64)])
def test_access_widths_agree(gm, interleaved, rot, d):
    """Tensors on 16, 8 and 2 bytes (and rotated parts of a multiple of 16, 8 and 2) take different accesses: the same
    bits, and the formula's."""
    B, Hq, Hkv, S = 2, 6, 3, 21
    gen = torch.Generator("cuda").manual_seed(rot + d)
    heads = Hq + 2 * Hkv
    src = torch.randn(B, S, heads, d, generator=gen, device="cuda").to(BF16)
    plan = gm.mercury_rope_init(rot, interleaved=interleaved)
    past = torch.tensor([5, 900], dtype=torch.int32, device="cuda")
    table = torch.randperm(2 * 60, generator=gen, device="cuda").to(torch.int32).reshape(2, 60)
    scale = torch.rand(Hkv, generator=gen, device="cuda") * 0.02 + 0.001
    got = []
    for off in (0, 4, 1):
        flat = torch.empty(src.numel() + 8, dtype=BF16, device="cuda")[off:off + src.numel()]
        x = flat.copy_(src.reshape(-1)).view(src.shape).transpose(1, 2)
        q, k, v = x.split([Hq, Hkv, Hkv], 1)
        res = [gm.mercury_rope(x, plan, start=40), gm.mercury_rope(x, plan, start=40, inverse=True)]
        for dtype, sc in ((BF16, None), (E4M3, scale)):
            kc, vc = (torch.zeros(120, Hkv, 16, d, device="cuda").to(dtype) for _ in range(2))
            qo = torch.empty(flat.numel() + 8, dtype=BF16, device="cuda")[off:off + B * S * Hq * d].view(B, S, Hq, d).transpose(1, 2)
            gm.mercury_kv_append(gm.PagedCache(kc, vc, table, k_scale=sc, v_scale=sc), k, v, past, rope=plan, q=q, q_out=qo)
            res += [bits(kc), bits(vc), qo]
        got.append(res)
    gm.mercury_sync_status()
    for res in got[1:]:
        for a, b in zip(got[0], res):
            assert torch.equal(a, b)
    x = src.transpose(1, 2)
    pos = (40 + torch.arange(S, device="cuda")).expand(B, S)
    ref = rotate(x, pos, frequencies(rot), interleaved)
    bound = rotation_bound(x, rot // 2, interleaved)
    assert_within(got[0][0], ref, bound + half_step(ref.abs() + bound, BF16), "rope")
    ref = rotate(x[:, :Hq], past[:, None].long() + torch.arange(S, device="cuda"), frequencies(rot), interleaved)
    bound = rotation_bound(x[:, :Hq], rot // 2, interleaved)
    assert_within(got[0][4], ref, bound + half_step(ref.abs() + bound, BF16), "q")


@pytest.mark.gpu
@pytest.mark.parametrize("rot,interleaved", [(24, False), (24, True), (40, True)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (0, 2), (3, 1)])
def test_few_heads_of_many_tokens(gm, Hq, Hkv, rot, interleaved):
    """A long prompt of few heads: the same bits as in short calls."""
    B, S, d = 2, 5003, 64
    gen = torch.Generator("cuda").manual_seed(rot + Hq)
    x = torch.randn(B, S, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(BF16).transpose(1, 2)
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    plan = gm.mercury_rope_init(rot, interleaved=interleaved)
    whole = gm.mercury_rope(x, plan, start=9)
    for s in range(0, S, 500):
        assert torch.equal(whole[:, :, s:s + 500], gm.mercury_rope(x[:, :, s:s + 500], plan, start=9 + s))
    table = torch.randperm(2 * 320, generator=gen, device="cuda").to(torch.int32).reshape(2, 320)
    past = torch.tensor([3, 77], dtype=torch.int32, device="cuda")
    for dtype in (BF16, E4M3):
        sc = torch.rand(Hkv, generator=gen, device="cuda") * 0.02 + 0.001 if dtype is E4M3 else None
        got = []
        for step in (S, 500):
            kc, vc = (torch.zeros(640, Hkv, 16, d, device="cuda").to(dtype) for _ in range(2))
            cache, qo = gm.PagedCache(kc, vc, table, k_scale=sc, v_scale=sc), torch.zeros_like(q) if Hq else None
            for s in range(0, S, step):
                part = slice(s, s + step)
                kw = dict(q=q[:, :, part], q_out=qo[:, :, part]) if Hq else {}
                gm.mercury_kv_append(cache, k[:, :, part], v[:, :, part], past + s, rope=plan, **kw)
            got.append([bits(kc), bits(vc)] + ([qo] if Hq else []))
        gm.mercury_sync_status()
        for a, b in zip(*got):
            assert torch.equal(a, b) and (a != 0).any()


@pytest.mark.gpu
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("scale", [1.0, 0.5, 3.0, 1 / 3, 0.7, -5.0, 1.1e-3, 2.0 ** -120, 1e-40, 2.0 ** 120, 0.0, math.inf, math.nan])
def test_append_stores_the_quotient(gm, scale, aligned):
    """Every bf16 value over a scale: the e4m3 nearest to the quotient's 32-bit rounding (ties to even), saturated;
    bit for bit, ties and their neighbours among them."""
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16).reshape(1, 1, 1024, 64)
    if not aligned:  # one element at a time
        y = torch.empty(1, 1, 1024, 65, dtype=BF16, device="cuda")[..., 1:]
        x = y.copy_(x)
    kc, vc = (torch.zeros(16, 1, 64, 64, device="cuda").to(E4M3) for _ in range(2))
    sc = torch.tensor([scale], device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda").reshape(1, 16)
    gm.mercury_kv_append(gm.PagedCache(kc, vc, table, k_scale=sc, v_scale=sc), x, x,
                         torch.zeros(1, dtype=torch.int32, device="cuda"))
    gm.mercury_sync_status()
    # the quotient in 64 bits, rounded to 32 (twice rounded, which is exact here: 8 by 24 bits), then by steps
    z = (x.double().cpu() / float(np.float32(scale)) if scale else x.double().cpu() / 0.0).float().double().reshape(-1)
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(2.0 ** -6, 448.0))) - 3)
    want = (torch.round(z.abs().clamp(max=512.0) / step) * step).clamp(max=448.0) * torch.sign(z)
    for cache in (kc, vc):
        got = cache.cpu().float().double().reshape(-1)
        nan = z.isnan()
        assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], want[~nan])


# ------------------------------------------------------------------------------- attention

def run_attention(gm, B, Hq, Hkv, Sq, d, page, lens, dtype=BF16, new=None, causal=True, bf16_out=False, scale=1.5,
                  seed=0, gap=0, spoil=None):
    gen = torch.Generator("cuda").manual_seed(seed)
    max_pages = max(1, -(-max(lens) // page)) + 1
    k_cache, v_cache, table, (ks, vs) = make_cache(B, Hkv, d, page, max_pages, dtype, gen, gap=gap)
    if spoil is not None:
        spoil(k_cache, v_cache, table)
    for b, n in enumerate(lens):  # entries behind a sequence's last page are never followed
        table[b, -(-n // page):] = -1
    q = (torch.randn(B, Hq, Sq, d, generator=gen, device="cuda") * scale).to(BF16)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    out = torch.full((B, Hq, Sq, d), 9.0, dtype=BF16 if bf16_out else FP32, device="cuda")
    lse = torch.full((B, Hq, Sq), 9.0, device="cuda")
    call = gm.mercury_attn_paged_bf16 if bf16_out else gm.mercury_attn_paged
    o, l = call(q, cache, lens_t, new_lens=new_t, causal=causal, out=out, lse=lse)
    gm.mercury_sync_status()
    assert o is out and l is lse
    return dict(q=q, k=k_cache, v=v_cache, table=table, ks=ks, vs=vs, out=out, lse=lse, cache=cache, lens=lens_t,
                new=new_t, call=call)


def check_attention(r, lens, new, causal, page):
    B, Hq, Sq, d = r["q"].shape
    for b in range(B):
        n = Sq if new is None else new[b]
        k, v = gather_states(r["k"], r["ks"], r["table"][b], lens[b]), gather_states(r["v"], r["vs"], r["table"][b], lens[b])
        limits = [lens[b] - n + i + 1 if causal else lens[b] for i in range(n)]
        o, l, eo, el = attention(r["q"][b, :, :n], k, v, limits)
        if r["out"].dtype is BF16:
            eo = eo + half_step(o.abs() + eo, BF16)
        assert_within(r["out"][b, :, :n], o, eo, "O of sequence %d" % b)
        assert_within(r["lse"][b, :, :n], l, el, "LSE of sequence %d" % b)
        assert (r["out"][b, :, n:] == 9.0).all() and (r["lse"][b, :, n:] == 9.0).all()


SHAPES = [
    # B, Hq, Hkv, Sq, d, page, lens
    (1, 1, 1, 1, 128, 16, [1]),
    (1, 8, 8, 1, 64, 16, [0]),
    (4, 8, 2, 1, 128, 16, [0, 1, 127, 129]),
    (5, 8, 1, 1, 64, 16, [255, 256, 257, 1, 1000]),
    (2, 32, 8, 1, 128, 16, [4096, 3333]),
    (1, 64, 8, 1, 128, 64, [20011]),
    (3, 6, 2, 1, 128, 7, [50, 6, 700]),
    (2, 3, 3, 1, 64, 1, [40, 129]),
    (2, 10, 2, 2, 128, 24, [30, 2]),          # 10 rows: one full tile
    (2, 16, 1, 1, 64, 32, [513, 90]),
    (3, 32, 8, 4, 128, 16, [4, 260, 3000]),   # 16 rows
    (2, 16, 2, 3, 64, 16, [3, 700]),          # 24 rows
    (2, 20, 1, 2, 128, 128, [2, 1500]),       # 40 rows: two row tiles
    (1, 4, 1, 64, 64, 16, [100]),             # 256 rows
    (2, 7, 7, 9, 128, 8, [9, 77]),
    (2, 128, 1, 1, 128, 16, [300, 5000]),     # 128 query heads on one
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("bf16_out", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,d,page,lens", SHAPES)
def test_paged_attention_matches_its_formula(gm, dtype, bf16_out, B, Hq, Hkv, Sq, d, page, lens):
    r = run_attention(gm, B, Hq, Hkv, Sq, d, page, lens, dtype, bf16_out=bf16_out, seed=sum(lens) + Hq)
    check_attention(r, lens, None, True, page)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_padded_batch(gm, dtype, causal):
    """Fewer new tokens in some sequences (none in one), fewer keys than new tokens, no keys at all."""
    lens, new = [500, 3, 40, 2, 0, 130], [4, 3, 0, 5, 2, 1]
    r = run_attention(gm, 6, 8, 2, 5, 128, 16, lens, dtype, new=new, causal=causal, seed=3)
    check_attention(r, lens, new, causal, 16)


@pytest.mark.gpu
def test_paged_attention_large_batches(gm):
    """More sequences than a block scans at once; whole runs of them without work."""
    gen = np.random.default_rng(5)
    B = 700
    lens = [int(x) for x in gen.integers(0, 200, B)]
    new = [int(x) for x in gen.integers(0, 2, B)]
    new[100:520] = [0] * 420
    r = run_attention(gm, B, 2, 1, 1, 64, 16, lens, new=new, seed=6)
    check_attention(r, lens, new, True, 16)
    r = run_attention(gm, 300, 1, 1, 1, 64, 16, [0] * 300, new=[0] * 300, seed=7)
    assert (r["out"] == 9.0).all() and (r["lse"] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pages_apart_and_shared(gm, dtype):
    """Pages as slices of a larger allocation, and a prefix that two sequences share."""
    def share(k, v, table):
        table[1, :3] = table[0, :3]
    r = run_attention(gm, 2, 8, 4, 1, 128, 16, [100, 70], dtype, gap=128, spoil=share, seed=8)
    check_attention(r, [100, 70], None, True, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_hidden_rows_do_not_matter(gm, dtype, value):
    """NaN and infinities (NaN alone in e4m3) in cache rows that no row, or only a later row, sees."""
    if dtype is E4M3 and value == math.inf:
        pytest.skip("e4m3 has no infinity")
    lens, B, Sq, page = [131, 64, 7, 300], 4, 4, 16

    def spoil(k, v, table):
        for c in (k, v):
            b8 = c.view(torch.uint8) if dtype is E4M3 else c
            bad = 0x7f if dtype is E4M3 else value
            for b, n in enumerate(lens):
                for at in list(range(n, (n + page - 1) // page * page)) + [n - 1, n - 2]:  # behind, and the last two tokens
                    b8[table[b, at // page].long(), :, at % page] = bad

    for Hq, Hkv in ((4, 2), (8, 2), (8, 1)):
        r = run_attention(gm, B, Hq, Hkv, Sq, 128, page, lens, dtype, spoil=spoil, seed=9)
        for b, n in enumerate(lens):
            k, v = gather_states(r["k"], r["ks"], r["table"][b], n - 2), gather_states(r["v"], r["vs"], r["table"][b], n - 2)
            o, l, eo, el = attention(r["q"][b, :, :2], k, v, [n - 3, n - 2])
            assert_within(r["out"][b, :, :2], o, eo, "O")
            assert_within(r["lse"][b, :, :2], l, el, "LSE")
            # what does see them says so
            assert not torch.isfinite(r["out"][b, :, 2:]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(2, 2, 5), (8, 2, 4), (8, 1, 4), (16, 2, 7), (16, 1, 64)])
def test_values_that_some_rows_see(gm, dtype, d, Hq, Hkv, Sq):
    """Single NaN (and infinite) elements among the new tokens' values: not finite in their column of the rows that
    see them, and nowhere else.  The new tokens lie across the ends of pages, of a warp's keys and of tiles."""
    lens, page = [Sq, 133, 257, 515, 1026], 16
    gen = torch.Generator("cpu").manual_seed(d + Hq)
    spots = []  # (sequence, key, head, column)

    def spoil(k, v, table):
        b8 = v.view(torch.uint8) if dtype is E4M3 else v
        for b, n in enumerate(lens):
            for i in range(0 if Sq < 64 else 3, Sq, 1 if Sq < 64 else 9):
                at, h, col = n - Sq + i, i % Hkv, int(torch.randint(0, d, (1,), generator=gen))
                spots.append((b, at, h, col))
                b8[table[b, at // page].long(), h, at % page, col] = 0x7f if dtype is E4M3 else (math.nan, math.inf)[i % 2]

    r = run_attention(gm, len(lens), Hq, Hkv, Sq, d, page, lens, dtype, spoil=spoil, seed=13)
    gm.mercury_sync_status()
    G = Hq // Hkv
    hit = torch.zeros_like(r["out"], dtype=torch.bool)
    for b, at, h, col in spots:
        hit[b, h * G:(h + 1) * G, max(at - (lens[b] - Sq), 0):, col] = True
    assert torch.equal(~torch.isfinite(r["out"]), hit)
    for b, n in enumerate(lens):
        k, v = gather_states(r["k"], r["ks"], r["table"][b], n), gather_states(r["v"], r["vs"], r["table"][b], n)
        v = torch.where(torch.isfinite(v), v, 0.0)
        o, l, eo, el = attention(r["q"][b], k, v, [n - Sq + i + 1 for i in range(Sq)])
        fine = ~hit[b]
        assert_within(r["out"][b][fine], o[fine], eo[fine], "O")
        assert_within(r["lse"][b], l, el, "LSE")


@pytest.mark.gpu
def test_extreme_scores(gm):
    """Scores far apart: one key takes everything, earlier and later than its rivals; tiny and huge queries."""
    for at, scale in ((0, 40.0), (999, 40.0), (500, 1e-30), (3, 0.0)):
        def spoil(k, v, table, at=at):
            k[table[0, at // 16].long(), :, at % 16] *= 8.0
        for dtype in (BF16, E4M3):
            r = run_attention(gm, 1, 4, 2, 1, 128, 16, [1000], dtype, scale=scale, spoil=spoil if dtype is BF16 else None, seed=at)
            check_attention(r, [1000], None, True, 16)


@pytest.mark.gpu
def test_results_do_not_change_between_calls(gm):
    r = run_attention(gm, 3, 32, 8, 1, 128, 16, [9000, 1, 4000], seed=12)
    for _ in range(3):
        out, lse = r["call"](r["q"], r["cache"], r["lens"])
        assert torch.equal(out, r["out"]) and torch.equal(lse, r["lse"])


@pytest.mark.gpu
def test_strided_queries(gm):
    r = run_attention(gm, 2, 8, 2, 3, 128, 16, [300, 33], seed=13)
    wide = torch.zeros(2, 3, 12, 128, dtype=BF16, device="cuda")
    q = wide.transpose(1, 2)[:, 2:10]
    q.copy_(r["q"])
    out, lse = gm.mercury_attn_paged(q, r["cache"], r["lens"])
    assert torch.equal(out, r["out"]) and torch.equal(lse, r["lse"])


# --------------------------------------------------------------------- streams, graphs, runs

@pytest.mark.gpu
def test_both_ways_into_a_call(gm):
    """A call goes through the C extension or, with a stream given, through the Python checks: the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(71)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen)
    here = torch.cuda.current_stream()
    plan = gm.mercury_rope_init(64)
    pos = torch.randint(-9, 9000, (2, 5), device="cuda", generator=gen, dtype=torch.int32)
    for x in (rand(2, 3, 5, 64), rand(2, 3, 5, 64).to(BF16), rand(2, 5, 3, 64).to(BF16).transpose(1, 2)):
        for p, start, inverse in ((None, 7, False), (pos, 0, True), (pos[0], 0, False)):
            a, b = torch.zeros_like(x), torch.zeros_like(x)
            assert gm.mercury_rope(x, plan, positions=p, start=start, inverse=inverse, out=a) is a
            gm.mercury_rope(x, plan, positions=p, start=start, inverse=inverse, out=b, stream=here)
            assert torch.equal(a, b) and not torch.equal(a, x)
    table = torch.randperm(8, device="cuda", generator=gen).to(torch.int32).reshape(2, 4)
    past = torch.tensor([3, 20], dtype=torch.int32, device="cuda")
    new = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    k, v = rand(2, 5, 2, 64).to(BF16).transpose(1, 2), rand(2, 2, 5, 64).to(BF16)
    q = rand(2, 4, 5, 64).to(BF16)
    for fresh in (None, new):
        for rope in (None, plan):
            got = []
            for stream in (None, here):
                cache = gm.PagedCache(torch.zeros(8, 2, 16, 64, dtype=BF16, device="cuda"),
                                      torch.zeros(8, 2, 16, 64, dtype=BF16, device="cuda"), table)
                qo = torch.zeros_like(q)
                assert gm.mercury_kv_append(cache, k, v, past, new_lens=fresh, rope=rope, q=q, q_out=qo, stream=stream) is qo
                assert gm.mercury_kv_append(cache, k, v, past, new_lens=fresh, rope=rope, stream=stream) is None
                res = [cache.k_cache, cache.v_cache, qo]
                for call, dtype in ((gm.mercury_attn_paged, FP32), (gm.mercury_attn_paged_bf16, BF16)):
                    out, lse = torch.zeros(q.shape, dtype=dtype, device="cuda"), torch.zeros(q.shape[:3], device="cuda")
                    res += call(qo, cache, past + 5, new_lens=fresh, causal=rope is None, out=out, lse=lse, stream=stream)
                    assert res[-1] is lse and res[-2] is out
                got.append(res)
            gm.mercury_sync_status()
            assert all(torch.equal(a, b) for a, b in zip(*got)) and all(a.abs().sum() > 0 for a in got[0])


@pytest.mark.gpu
def test_streams_and_graphs(gm):
    """Calls on a side stream, two calls at once on two streams, and captured graphs that share the cache."""
    r = run_attention(gm, 4, 32, 8, 1, 128, 16, [5000, 1, 2500, 129], seed=14)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append(gm.mercury_attn_paged(r["q"], r["cache"], r["lens"]))
    outs.append(gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], stream=s1))
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, r["out"]) and torch.equal(lse, r["lse"])
    graphs, got = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        o, l = torch.zeros_like(r["out"]), torch.zeros_like(r["lse"])
        with torch.cuda.graph(g):
            gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], out=o, lse=l)
        graphs.append(g)
        got.append((o, l))
    r["lens"].copy_(torch.tensor([77, 5000, 4, 0], device="cuda"))  # lengths are read when the graph runs
    r["table"][:, :313] = torch.arange(4 * 313, device="cuda", dtype=torch.int32).view(4, 313)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    out, lse = gm.mercury_attn_paged(r["q"], r["cache"], r["lens"])
    gm.mercury_sync_status()
    for o, l in got:
        assert torch.equal(o, out) and torch.equal(l, lse)
    r.update(out=out, lse=lse)
    check_attention(r, [77, 5000, 4, 0], None, True, 16)


@pytest.mark.gpu
def test_two_threads_at_once(gm):
    """Two host threads with a stream and a cache each, calling at the same time (a call leaves the interpreter while it
    launches): the results of one after the other."""
    plan = gm.mercury_rope_init(128)

    def inputs(seed):
        gen = torch.Generator("cuda").manual_seed(seed)
        B, Hq, Hkv, page = 3, 8, 2, 16
        k_cache, v_cache, table, _ = make_cache(B, Hkv, 128, page, 40, BF16, gen)
        rand = lambda h: torch.randn(B, h, 1, 128, generator=gen, device="cuda").to(BF16)
        past = torch.randint(1, 600, (B,), generator=gen, device="cuda").to(torch.int32)
        return gm.PagedCache(k_cache, v_cache, table), rand(Hq), rand(Hkv), rand(Hkv), past

    def steps(data, stream, n=40):
        cache, q, k, v, past = data
        with torch.cuda.stream(stream):
            past, res = past.clone(), []
            for _ in range(n):
                qo, out, lse = torch.empty_like(q), torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
                gm.mercury_kv_append(cache, k, v, past, rope=plan, q=q, q_out=qo)
                past += 1
                gm.mercury_attn_paged(qo, cache, past, out=out, lse=lse)
                res.append((gm.mercury_rope(qo, plan, inverse=True, out=qo), out, lse))
            return res

    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [steps(inputs(s), streams[0]) for s in (1, 2)]
    data = [inputs(s) for s in (1, 2)]
    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        got = list(pool.map(steps, data, streams))
    torch.cuda.synchronize()
    gm.mercury_sync_status()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert all(torch.equal(i, j) for i, j in zip(x, y))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_a_prompt_and_its_continuation(gm, dtype):
    """The operators as a serving loop runs them: a ragged batch of prompts goes into the cache while their own
    attention runs on rotated heads, then tokens follow one by one and once three at a time, as a captured step."""
    B, Hq, Hkv, d, page, S = 3, 8, 2, 128, 16, 96
    gen = torch.Generator("cuda").manual_seed(21)
    k_cache, v_cache, table, (ks, vs) = make_cache(B, Hkv, d, page, 8, dtype, gen)
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    freq = frequencies(d)
    plan = gm.mercury_rope_init(d)
    prompt = [96, 40, 1]
    steps = [(torch.randn(B, S, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(BF16), prompt)]
    for n in (1, 1, 3, 1):
        steps.append((torch.randn(B, n, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(BF16), [n] * B))
    lens = [0] * B
    for x, new in steps:
        n = x.shape[1]
        q, k, v = x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
        past = torch.tensor(lens, dtype=torch.int32, device="cuda")
        new_t = torch.tensor(new, dtype=torch.int32, device="cuda")
        q_rot = gm.mercury_kv_append(cache, k, v, past, new_lens=new_t, rope=plan, q=q)
        lens = [a + b for a, b in zip(lens, new)]
        if n == S:
            # the first prompt is as long as the padding: its own attention by the prompt path
            k_rot = gm.mercury_rope(k[:1], plan)
            o1, l1 = gm.mercury_attn_sharded(q_rot[:1].contiguous(), k_rot, v[:1].contiguous(), 4, 1, True)
            ref = attention(q_rot[0], k_rot[0].double(), v[0].double(), [i + 1 for i in range(S)])
            assert (o1[0].double() - ref[0]).abs().max() <= 2e-2 and (l1[0].double() - ref[1]).abs().max() <= 1e-3
            continue
        lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out, lse = gm.mercury_attn_paged(q_rot, cache, lens_t)
        gm.mercury_sync_status()
        for b in range(B):
            qr = rotate(q[b:b + 1], past[b:b + 1, None] + torch.arange(n, device="cuda"), freq, False)[0]
            assert_within(q_rot[b], qr, half_step(qr, BF16) + rotation_bound(q[b], d // 2, False), "rotated q")
            kk, vv = gather_states(k_cache, ks, table[b], lens[b]), gather_states(v_cache, vs, table[b], lens[b])
            o, l, eo, el = attention(q_rot[b], kk, vv, [lens[b] - n + i + 1 for i in range(n)])
            assert_within(out[b], o, eo, "O")
            assert_within(lse[b], l, el, "LSE")
        # the parts of a context: paged over the newest page's worth, merged with the rest
    # a decode step as one captured graph: append, then attention
    x = torch.randn(B, 1, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(BF16)
    q, k, v = x.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
    past = torch.tensor(lens, dtype=torch.int32, device="cuda")
    total = past + 1
    q_rot, out, lse = torch.zeros(B, Hq, 1, d, dtype=BF16, device="cuda"), torch.zeros(B, Hq, 1, d, device="cuda"), torch.zeros(B, Hq, 1, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gm.mercury_kv_append(cache, k, v, past, rope=plan, q=q, q_out=q_rot)
        gm.mercury_attn_paged(q_rot, cache, total, out=out, lse=lse)
    g.replay()
    torch.cuda.synchronize()
    o2, l2 = gm.mercury_attn_paged(q_rot, cache, total)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    kk, vv = gather_states(k_cache, ks, table[0], lens[0] + 1), gather_states(v_cache, vs, table[0], lens[0] + 1)
    o, l, eo, el = attention(q_rot[0], kk, vv, [lens[0] + 1])
    assert_within(out[0], o, eo, "O of the captured step")


@pytest.mark.gpu
def test_parts_of_a_context_merge(gm):
    """(O, LSE) over a paged part and over a dense shard join by the log-sum-exp merge into the whole."""
    gen = torch.Generator("cuda").manual_seed(31)
    Hq, Hkv, d, n1, n2 = 8, 2, 128, 512, 77
    k1, v1 = (torch.randn(1, Hkv, n1, d, generator=gen, device="cuda").to(BF16) for _ in (0, 1))
    k_cache, v_cache, table, _ = make_cache(1, Hkv, d, 16, 5, BF16, gen)
    q = torch.randn(1, Hq, 1, d, generator=gen, device="cuda").to(BF16)
    o1, l1 = gm.mercury_attn_decode(q, k1, v1)
    o2, l2 = gm.mercury_attn_paged(q, gm.PagedCache(k_cache, v_cache, table),
                                   torch.tensor([n2], dtype=torch.int32, device="cuda"))
    out, lse = gm.mercury_lse_merge(torch.stack([o1, o2]), torch.stack([l1, l2]))
    gm.mercury_sync_status()
    k = torch.cat([k1[0].double(), gather_states(k_cache, None, table[0], n2)], 1)
    v = torch.cat([v1[0].double(), gather_states(v_cache, None, table[0], n2)], 1)
    o, l, _, _ = attention(q[0], k, v, [n1 + n2])
    assert (out[0].double() - o).abs().max() <= 2e-2 and (lse[0].double() - l).abs().max() <= 1e-3


@pytest.mark.gpu
def test_long_offsets(gm):
    """A cache whose pages lie beyond 2^31 elements."""
    n, Hkv, page, d = 1100, 16, 1024, 128  # 2.3e9 elements a tensor
    k_cache = torch.empty(n, Hkv, page, d, dtype=BF16, device="cuda")
    v_cache = torch.empty_like(k_cache)
    gen = torch.Generator("cuda").manual_seed(41)
    table = torch.tensor([[n - 1, 0], [n - 2, n - 3]], dtype=torch.int32, device="cuda")
    for p in (0, n - 1, n - 2, n - 3):
        for c in (k_cache, v_cache):
            c[p] = torch.randn(Hkv, page, d, generator=gen, device="cuda").to(BF16)
    cache = gm.PagedCache(k_cache, v_cache, table)
    x = torch.randn(3, 2, Hkv, 1, d, generator=gen, device="cuda").to(BF16)
    lens = [1030, 2000]
    past = torch.tensor([a - 1 for a in lens], dtype=torch.int32, device="cuda")
    q = gm.mercury_kv_append(cache, x[1], x[2], past, rope=gm.mercury_rope_init(d), q=x[0])
    out, lse = gm.mercury_attn_paged(q, cache, past + 1)
    gm.mercury_sync_status()
    r = dict(q=q, k=k_cache, v=v_cache, table=table, ks=None, vs=None, out=out, lse=lse)
    check_attention(r, lens, None, True, page)
    ref = rotate(x[1], past[:, None], frequencies(d), False)
    for b in range(2):
        got = k_cache[table[b, (lens[b] - 1) // page].long(), :, (lens[b] - 1) % page]
        assert_within(got, ref[b, :, 0], half_step(ref[b, :, 0], BF16) + rotation_bound(x[1], 64, False)[b, :, 0], "key")


# ----------------------------------------------------------------- checked on the device

@pytest.mark.gpu
def test_binding_refusals_on_the_device(gm):
    c = torch.zeros(4, 2, 16, 64, dtype=BF16, device="cuda")
    t = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    PC = gm.PagedCache
    with pytest.raises(TypeError, match="bfloat16"):
        PC(c.half(), c.half(), t)
    with pytest.raises(ValueError, match="num_pages"):
        PC(c, c[:3], t)
    with pytest.raises(ValueError, match="contiguous"):
        PC(c.transpose(1, 2), c.transpose(1, 2), t)
    with pytest.raises(ValueError, match="equally far"):
        PC(c, torch.zeros(4, 3, 16, 64, dtype=BF16, device="cuda")[:, :2], t)
    with pytest.raises(TypeError, match="int32"):
        PC(c, c, t.long())
    with pytest.raises(ValueError, match="block_table"):
        PC(c, c, t[0])
    with pytest.raises(ValueError, match="needs k_scale"):
        PC(c.to(E4M3), c.to(E4M3), t)
    with pytest.raises(ValueError, match="e4m3"):
        PC(c, c, t, k_scale=torch.ones(2, device="cuda"))
    cache = PC(c, c.clone(), t)
    q = torch.zeros(2, 4, 1, 64, dtype=BF16, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    for bad in (q[:1], q[..., :32], q[0]):
        with pytest.raises(ValueError):
            gm.mercury_attn_paged(bad, cache, lens)
    with pytest.raises(TypeError):
        gm.mercury_attn_paged(q.float(), cache, lens)
    with pytest.raises(TypeError):
        gm.mercury_attn_paged(q, cache, lens.long())
    with pytest.raises(TypeError):
        gm.mercury_attn_paged(q, cache, None)
    with pytest.raises(ValueError, match="shape"):
        gm.mercury_attn_paged(q, cache, lens[:1])
    with pytest.raises(ValueError, match="out must have"):
        gm.mercury_attn_paged(q, cache, lens, out=torch.zeros(2, 4, 1, 32, device="cuda"))
    with pytest.raises(gm.MercuryError):
        gm.mercury_attn_paged(q[:, :3], cache, lens)
    k = torch.zeros(2, 2, 3, 64, dtype=BF16, device="cuda")
    for bad in (k[:1], k[:, :1], k[..., :32], k[0]):
        with pytest.raises(ValueError):
            gm.mercury_kv_append(cache, bad, bad, lens)
    with pytest.raises(ValueError):
        gm.mercury_kv_append(cache, k, k[:, :, :2], lens)
    with pytest.raises(ValueError, match="q_out without q"):
        gm.mercury_kv_append(cache, k, k, lens, q_out=q)
    with pytest.raises(TypeError):
        gm.mercury_kv_append(cache, k, k, None)
    with pytest.raises(gm.MercuryError, match="overlap"):
        gm.mercury_rope(k, gm.mercury_rope_init(64), out=torch.zeros(2, 1, 3, 64, dtype=BF16, device="cuda").expand(2, 2, 3, 64))


@pytest.mark.gpu
def test_pages_and_lengths_out_of_range_are_reported(gm):
    """The kernels test every page, position and length; a bad one is skipped and reported, the rest is right."""
    r = run_attention(gm, 3, 4, 2, 1, 128, 16, [100, 60, 90], seed=51)
    keep = r["out"].clone(), r["lse"].clone()

    def expect(fn):
        fn()
        with pytest.raises(gm.MercuryError) as e:
            gm.mercury_sync_status()
        assert e.value.status == gm.MERCURY_EBOUNDS
        gm.mercury_sync_status()

    good = r["table"].clone()
    for entry in (-1, r["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        r["table"][1, 2] = entry
        expect(lambda: gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], out=r["out"], lse=r["lse"]))
        for b in (0, 2):
            assert torch.equal(r["out"][b], keep[0][b]) and torch.equal(r["lse"][b], keep[1][b])
        assert torch.isfinite(r["out"]).all()
    r["table"].copy_(good)
    for n in (-3, 10 ** 6, 2 ** 31 - 1):
        bad = torch.tensor([100, n, 90], dtype=torch.int32, device="cuda")
        expect(lambda: gm.mercury_attn_paged(r["q"], r["cache"], bad, out=r["out"], lse=r["lse"]))
        for b in (0, 2):
            assert torch.equal(r["out"][b], keep[0][b])
    expect(lambda: gm.mercury_attn_paged(r["q"], r["cache"], r["lens"], new_lens=torch.tensor([1, 2, -1], dtype=torch.int32, device="cuda")))

    k = torch.ones(3, 2, 2, 128, dtype=BF16, device="cuda")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    for past in ([0, -1, 5], [0, 16 * r["table"].shape[1] - 1, 5], [0, 2 ** 31 - 1, 5], [0, -2 ** 31, 5]):
        kc, vc = r["k"].clone(), r["v"].clone()
        cache = gm.PagedCache(kc, vc, good.clamp(min=0))
        expect(lambda: gm.mercury_kv_append(cache, k, k, torch.tensor(past, dtype=torch.int32, device="cuda")))
        assert (kc[good[0, 0].long(), :, :2] == 1).all() and (vc[good[2, 0].long(), :, 5:7] == 1).all()
    expect(lambda: gm.mercury_kv_append(cache, k, k, zero, new_lens=torch.tensor([2, 3, -1], dtype=torch.int32, device="cuda")))
    cache.block_table[1, 0] = kc.shape[0]
    expect(lambda: gm.mercury_kv_append(cache, k, k, zero))


@pytest.mark.gpu
def test_a_copy_that_never_comes_ends_in_a_timeout(gm, monkeypatch):
    """With one copy withheld (the test hook) its wait runs out, the status says so, and the next call is right."""
    lens = [700, 20]
    r = run_attention(gm, 2, 8, 2, 1, 128, 16, lens, seed=61)
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
