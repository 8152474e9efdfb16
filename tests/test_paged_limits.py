"""The serving operators where their promises are hardest to keep: outputs that a call makes for another stream,
values that are not finite beside one another, sums over long contexts, weights far below the largest, copies that
never come.

Bounds are derived where they are used; a rounding is off by at most half a step, as in test_paged.py, whose 64-bit
definitions these tests share.
"""
import contextlib
import ctypes
import importlib.util
import math
import subprocess
import sys
import sysconfig
import time
import types

import pytest
import torch

from tests.conftest import ROOT
from tests.test_paged import (BF16, E4M3, FP32, assert_within, attention, cache_struct, gather_states,
                              gm, m, make_cache)  # noqa: F401  (gm, m: fixtures)


# --------------------------------------------------------- outputs that a call makes itself

class _Tensor:
    """As much of a CUDA tensor as the Python side of a call looks at."""

    def __init__(self, shape, dtype, made_on=None):
        self.shape, self.dtype, self.made_on, self.kept_for = torch.Size(shape), dtype, made_on, []

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000

    def record_stream(self, stream):
        self.kept_for.append(stream)

    device = "cuda:0"


@pytest.fixture
def pretend(m, monkeypatch):
    """A device on which nothing runs: the current stream is 7, and every output says on which it was made."""
    active = [7]

    @contextlib.contextmanager
    def context(stream):
        active.append(stream)
        yield
        active.pop()

    make = lambda shape, dtype, device: _Tensor(shape, dtype, active[-1])  # noqa: E731
    names = types.SimpleNamespace(Tensor=_Tensor, empty=make, zeros=make, bf16=BF16, fp32=FP32, int32=torch.int32,
                                  current_device=lambda: 0, raw_stream=lambda dev: 7, stream_context=context,
                                  external_stream=lambda ptr, device: ptr, current_stream=lambda dev: 7)
    ran_on = []
    call = lambda *a: ran_on.append(a[-1]) or 0  # noqa: E731
    monkeypatch.setattr(m, "_torch_names", names)
    monkeypatch.setattr(m, "lib", types.SimpleNamespace(mercury_rope=call, mercury_kv_append=call,
                                                        mercury_attn_paged=call, mercury_attn_paged_bf16=call))
    cache = m.PagedCache.__new__(m.PagedCache)
    cache.struct = cache_struct(m)
    cache.B, cache.Hkv, cache.d, cache.device_index, cache._ref, cache.address = 2, 2, 128, 0, None, 0
    return types.SimpleNamespace(m=m, cache=cache, ran_on=ran_on)


@pytest.mark.parametrize("stream", [None, 7, 9])
@pytest.mark.parametrize("padded", [False, True])
def test_own_outputs_are_made_on_the_stream_of_the_call(pretend, stream, padded):
    """Zeros that another stream writes could land behind the kernel's rows."""
    m, cache = pretend.m, pretend.cache
    t = lambda *shape, dtype=BF16: _Tensor(shape, dtype)  # noqa: E731
    lens = t(2, dtype=torch.int32)
    kw = dict(new_lens=lens if padded else None, stream=stream)
    made = list(m.mercury_attn_paged(t(2, 4, 3, 128), cache, lens, **kw))
    made += m.mercury_attn_paged_bf16(t(2, 4, 3, 128), cache, lens, **kw)
    made.append(m.mercury_kv_append(cache, t(2, 2, 3, 128), t(2, 2, 3, 128), lens, q=t(2, 4, 3, 128), **kw))
    made.append(m.mercury_rope(t(2, 4, 3, 128), m.RopePlan(), stream=stream))
    where = 7 if stream is None else stream
    assert pretend.ran_on == [where] * 4
    assert [x.made_on for x in made] == [where] * 6
    # on another stream than the caller's, not reused before the caller's work on it is done
    assert all(x.kept_for == ([7] if where == 9 else []) for x in made)


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [False, True])
def test_padded_calls_on_a_given_stream_keep_their_rows(gm, as_int):
    """The caller's own stream is busy for some milliseconds while a call runs on another one: its outputs are whole."""
    gen = torch.Generator("cuda").manual_seed(3)
    B, Hq, Hkv, S, d = 3, 8, 2, 4, 64
    k_cache, v_cache, table, _ = make_cache(B, Hkv, d, 16, 4, BF16, gen)
    cache = gm.PagedCache(k_cache, v_cache, table)
    rand = lambda h: torch.randn(B, h, S, d, generator=gen, device="cuda").to(BF16)  # noqa: E731
    q, k, v = rand(Hq), rand(Hkv), rand(Hkv)
    past = torch.tensor([3, 20, 40], dtype=torch.int32, device="cuda")
    new = torch.tensor([4, 2, 1], dtype=torch.int32, device="cuda")
    plan, pos = gm.mercury_rope_init(d), torch.arange(5, 5 + S, dtype=torch.int32, device="cuda")
    total = past + new
    zero = torch.zeros_like(q), torch.zeros(q.shape, device="cuda"), torch.zeros(q.shape[:3], device="cuda")
    want = [gm.mercury_kv_append(cache, k, v, past, new_lens=new, rope=plan, q=q, q_out=zero[0])]
    want += gm.mercury_attn_paged(want[0], cache, total, new_lens=new, out=zero[1], lse=zero[2])
    want.append(gm.mercury_rope(q, plan, pos))
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # what follows on this stream waits
    got = [gm.mercury_kv_append(cache, k, v, past, new_lens=new, rope=plan, q=q, stream=stream)]
    got += gm.mercury_attn_paged(got[0], cache, total, new_lens=new, stream=stream)
    got.append(gm.mercury_rope(q, plan, pos, stream=stream))
    torch.cuda.synchronize()
    gm.mercury_sync_status()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ sums over long contexts

def shared_cache(gm, n, d, dtype, gen, B):
    """One sequence of n tokens whose pages B sequences name: jobs for every SM in little memory."""
    page = 64
    k_cache, v_cache, table, (ks, vs) = make_cache(1, 1, d, page, -(-n // page), dtype, gen)
    return gm.PagedCache(k_cache, v_cache, table.expand(B, -1).contiguous(), k_scale=ks, v_scale=vs)


def states(cache, n):
    return (gather_states(c, s, cache.block_table[0], n)
            for c, s in ((cache.k_cache, cache.k_scale), (cache.v_cache, cache.v_scale)))


def sum_bound(n):
    """Relative bound of a sum of n weighted values that do not cancel, kept in 32 bits and rounded to nearest.

    Sixteen keys at a time, n/16 additions, each off by at most 2^-24 of the sum, independently and either way: beyond
    7 (n/16)^(1/2) 2^-24 the chance is 2 exp(-98) (Hoeffding).  A weight's exponent, at most 16 in powers of two, is
    off by 2^-21 and by 3 roundings of a factor, its exponential by 2^-22, its terms by 2^-23: 30 * 2^-24 in all, once
    above and once below the line, and a dozen joins and the quotient."""
    return (7 * math.sqrt(n) / 4 + 72) * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 16, 28, 64])
def test_sums_over_a_long_context(gm, dtype, d, rows):
    """32K keys whose values are all positive: the rounding of the sums shows, and nothing cancels."""
    n, B = 32768, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator("cuda").manual_seed(rows + d)
    cache = shared_cache(gm, n, d, dtype, gen, B)
    # scores of one product each, exact in 32 bits: multiples of 1/8 in [-2, 2] times multiples of 1/16 in [8, 12)
    scores = torch.randint(-16, 17, cache.k_cache.shape, generator=gen, device="cuda") / 8
    scores[..., 1:] = 0
    cache.k_cache.copy_(scores.to(dtype))
    cache.v_cache.copy_((cache.v_cache.float().abs() + (20 if dtype is E4M3 else 1)).clamp(max=448).to(dtype))
    if dtype is E4M3:
        cache.k_scale.fill_(1.0)
    q = torch.zeros(B, rows, 1, d, dtype=BF16, device="cuda")
    q[..., 0] = 8 + torch.arange(rows, device="cuda")[:, None] / 16
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out, lse = gm.mercury_attn_paged(q, cache, lens)
    gm.mercury_sync_status()
    k, v = states(cache, n)
    o, l, _, _ = attention(q[0], k, v, [n])
    assert ((out[0].double() - o) / o).abs().max() <= sum_bound(n)
    assert ((out.double() - o) / o).abs().max() <= sum_bound(n)  # the others' keys, cut elsewhere
    assert (lse.double() - l).abs().max() <= 72 * 2.0 ** -24 + 2.0 ** -22 * l.abs().max()


def sink(gm, dtype, rows, below, n=16384, d=128):
    """One key far above n - 1 equal ones, its value zero: all of O comes from weights e^-below of the largest.
    Returns O's relative error, LSE's error and the bound of a score (2^-21, as in attention())."""
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    cache = shared_cache(gm, n, d, dtype, torch.Generator("cuda").manual_seed(rows), B)
    if dtype is E4M3:
        cache.k_scale.fill_(1.0)
        cache.v_scale.fill_(1.0)
    first = cache.block_table[0, 0].long()
    k, v = torch.zeros(cache.k_cache.shape, device="cuda"), cache.v_cache.float().abs() % 1 + 1
    k[first, 0, 0, 0] = 1
    v[first, 0, 0] = 0
    cache.k_cache.copy_(k.to(dtype))
    cache.v_cache.copy_(v.to(dtype))
    q = torch.zeros(B, rows, 1, d, dtype=BF16, device="cuda")
    q[..., 0] = below * math.sqrt(d)
    out, lse = gm.mercury_attn_paged(q, cache, torch.full((B,), n, dtype=torch.int32, device="cuda"))
    gm.mercury_sync_status()
    o, l, _, _ = attention(q[0], *states(cache, n), [n])
    return ((out.double() - o) / o).abs().max().item(), (lse.double() - l).abs().max().item(), 2.0 ** -21 * below


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 16, 40])
@pytest.mark.parametrize("below", [8.0, 14.0, 17.0, 20.0])
def test_small_weights_beside_a_large_one(gm, rows, below):
    off, off_lse, ds = sink(gm, BF16, rows, below)
    assert off <= sum_bound(16384) + 2 * ds
    assert off_lse <= 72 * 2.0 ** -24 + ds


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 16, 40])
@pytest.mark.parametrize("below", [8.0, 12.0, 14.0, 17.0, 20.0])
def test_small_weights_beside_a_large_one_in_8_bits(gm, rows, below):
    """Weights enter the products as 16-bit terms, which hold the smallest ones to 2^-48 of the largest."""
    off, off_lse, ds = sink(gm, E4M3, rows, below)
    assert off <= sum_bound(16384) + 2 * ds + 2.0 ** -48 * math.exp(below)
    assert off_lse <= 72 * 2.0 ** -24 + ds


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 16, 28])
def test_scores_that_rise_slowly(gm, dtype, rows):
    """Each key a little above the last, up and down again: the maximum that the weights are taken relative to is
    behind the scores by as much as the kernel lets it be, and is raised many times."""
    n, d, page = 1500, 128, 64
    gen = torch.Generator("cuda").manual_seed(rows)
    cache = shared_cache(gm, n, d, dtype, gen, 3)
    at = torch.arange(n, device="cuda")
    wave = 40.0 * (1 - (at / 750.0 - 1).abs())
    k = torch.zeros(cache.k_cache.shape, device="cuda")
    k[cache.block_table[0][at // page].long(), 0, at % page, 0] = wave
    cache.k_cache.copy_(k.to(dtype))
    if dtype is E4M3:
        cache.k_scale.fill_(1.0)
    q = torch.zeros(3, rows, 1, d, dtype=BF16, device="cuda")
    q[..., 0] = math.sqrt(d)
    lens = torch.full((3,), n, dtype=torch.int32, device="cuda")
    out, lse = gm.mercury_attn_paged(q, cache, lens)
    gm.mercury_sync_status()
    o, l, eo, el = attention(q[0], *states(cache, n), [n])
    for b in range(3):
        assert_within(out[b], o, eo, "O")
        assert_within(lse[b], l, el, "LSE")


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Sq", [(2, 4), (4, 4), (6, 4), (8, 4), (7, 9), (40, 3)])
def test_whole_tokens_that_are_not_finite(gm, dtype, d, Hq, Sq):
    """Every value of the newer drafted tokens NaN (or infinite, turn by turn): several elements of a word, for one to
    four row groups of a tile and for two tiles.  Rows before such a token do not meet it, in any of many calls."""
    page, B = 16, 40
    gen = torch.Generator("cuda").manual_seed(Sq + d)
    lens = [200 + 17 * b for b in range(B)]
    k_cache, v_cache, table, (ks, vs) = make_cache(B, 1, d, page, -(-max(lens) // page), dtype, gen)
    b8 = v_cache.view(torch.uint8) if dtype is E4M3 else v_cache
    row = torch.full((d,), 0x7f, dtype=torch.uint8, device="cuda") if dtype is E4M3 else \
        torch.tensor([math.nan, math.inf, -math.inf], device="cuda").repeat(d)[:d].to(BF16)
    good = [b % Sq for b in range(B)]  # rows that see finite values only
    for b, n in enumerate(lens):
        for at in range(n - Sq + good[b], n):
            b8[table[b, at // page].long(), 0, at % page] = row
    q = torch.randn(B, Hq, Sq, d, generator=gen, device="cuda").to(BF16)
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = gm.mercury_attn_paged(q, cache, lens_t)
    gm.mercury_sync_status()
    for b, n in enumerate(lens):
        k = gather_states(k_cache, ks, table[b], n)
        v = gather_states(v_cache, vs, table[b], n - Sq + good[b])
        if good[b]:
            o, l, eo, el = attention(q[b, :, :good[b]], k[:, :v.shape[1]], v, [n - Sq + i + 1 for i in range(good[b])])
            assert_within(out[b, :, :good[b]], o, eo, "O of sequence %d" % b)
            assert_within(lse[b, :, :good[b]], l, el, "LSE of sequence %d" % b)
        assert not torch.isfinite(out[b, :, good[b]:]).any()
    same = torch.isfinite(out)
    for _ in range(30):
        again, lse2 = gm.mercury_attn_paged(q, cache, lens_t)
        assert torch.equal(torch.isfinite(again), same) and torch.equal(again[same], out[same]) and torch.equal(lse2, lse)
    gm.mercury_sync_status()


# ----------------------------------------------------------------------- pages and copies

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 8), (64, 64), (128, 256), (128, 7)])
def test_pages_outside_the_cache_count_as_zeros(gm, dtype, d, page):
    """Keys and values of zero, for every lane that finds such a page: single pages, neighbours, a whole tile of them."""
    B, Hq, n = 30, 4, 1500
    gen = torch.Generator("cuda").manual_seed(page)
    k_cache, v_cache, table, (ks, vs) = make_cache(B, 1, d, page, -(-n // page), dtype, gen)
    wrong = torch.rand(table.shape, generator=gen, device="cuda") < torch.linspace(0, 1, B, device="cuda")[:, None]
    table[wrong] = torch.randint(0, 2, (int(wrong.sum()),), generator=gen, device="cuda", dtype=torch.int32) * 2 ** 30 - 1
    cache = gm.PagedCache(k_cache, v_cache, table, k_scale=ks, v_scale=vs)
    q = torch.randn(B, Hq, 1, d, generator=gen, device="cuda").to(BF16)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for _ in range(5):
        out, lse = gm.mercury_attn_paged(q, cache, lens)
        with pytest.raises(gm.MercuryError) as e:
            gm.mercury_sync_status()
        assert e.value.status == gm.MERCURY_EBOUNDS
        zero = wrong.repeat_interleave(page, 1)[:, None, :n, None]
        for b in range(B):
            k, v = (gather_states(c, s, table[b].clamp(0, k_cache.shape[0] - 1), n).masked_fill(zero[b], 0.0)
                    for c, s in ((k_cache, ks), (v_cache, vs)))
            o, l, eo, el = attention(q[b], k, v, [n])
            assert_within(out[b], o, eo, "O of sequence %d" % b)
            assert_within(lse[b], l, el, "LSE of sequence %d" % b)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [64, 8, 7])
@pytest.mark.parametrize("rows", [4, 40])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_a_long_call_whose_copies_never_come_ends(gm, monkeypatch, dtype, rows, page):
    """Far more tiles a block than are ever on their way: a wait runs out, the block sends nothing more and ends when
    what it had sent has landed, the status says so, and the next call is right."""
    n, d, B = 4000, 128, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator("cuda").manual_seed(page)
    k_cache, v_cache, table, (ks, vs) = make_cache(1, 1, d, page, -(-n // page), dtype, gen)
    cache = gm.PagedCache(k_cache, v_cache, table.expand(B, -1).contiguous(), k_scale=ks, v_scale=vs)
    q = torch.randn(B, rows, 1, d, generator=gen, device="cuda").to(BF16)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    want = gm.mercury_attn_paged(q, cache, lens)
    gm.mercury_sync_status()
    for _ in range(2):
        with monkeypatch.context() as mp:
            mp.setenv("MERCURY_FAULT", "drop_page_copy")
            mp.setenv("MERCURY_WAIT_NS", "20000000")
            began = time.monotonic()
            gm.mercury_attn_paged(q, cache, lens)
            with pytest.raises(gm.MercuryError) as e:
                gm.mercury_sync_status()
            assert e.value.status == gm.MERCURY_ETIMEOUT
            assert time.monotonic() - began < 5  # 20 ms, not 20 ms a tile
        out, lse = gm.mercury_attn_paged(q, cache, lens)
        gm.mercury_sync_status()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# -------------------------------------------------------------------- the C side's build

def test_an_extension_belongs_to_one_interpreter(m, monkeypatch, tmp_path):
    """One built for another Python, next to this one's and newer than its source, is neither reused nor loaded."""
    from long_context_sharded_gb300 import build

    def for_abi(suffix):
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: suffix if name == "EXT_SUFFIX" else None)
        spec = importlib.util.spec_from_file_location("build_for_abi", build.__file__)
        b = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(b)
        monkeypatch.undo()
        return b

    assert m._build.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    one, other = for_abi(".cpython-398-a.so"), for_abi(".cpython-399-b.so")
    for b in (one, other):
        b.LIB_DIR = str(tmp_path)
        b.BINDING_PATH = str(tmp_path / b.BINDING_PATH.rsplit("/", 1)[1])
    with open(one.BINDING_PATH, "w") as f:
        f.write("another interpreter's")
    assert one.build_binding() == one.BINDING_PATH  # newer than its source
    made = other.build_binding()
    assert made == other.BINDING_PATH != one.BINDING_PATH
    with open(made, "rb") as f:
        assert f.read(4) == b"\x7fELF"


# ------------------------------------------------------------------------------- reports

@pytest.mark.gpu
def test_each_report_names_its_own_site(gm):
    """The status names where the first error since the last report was found, and forgets it."""
    gen = torch.Generator("cuda").manual_seed(1)
    k_cache, v_cache, table, _ = make_cache(2, 1, 64, 16, 4, BF16, gen)
    cache = gm.PagedCache(k_cache, v_cache, table)
    good = table.clone()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros(2, 1, 1, 64, dtype=BF16, device="cuda")

    def wrong_page(fn):
        table[1] = -1
        fn()
        table.copy_(good)

    attn = lambda lens, **kw: gm.mercury_attn_paged(q, cache, lens, **kw)  # noqa: E731
    append = lambda past, **kw: gm.mercury_kv_append(cache, q, q, past, **kw)  # noqa: E731
    cases = [("0x901", lambda: attn(ints(3, -1))), ("0x902", lambda: attn(ints(3, 4), new_lens=ints(1, 2))),
             ("0x903", lambda: wrong_page(lambda: attn(ints(3, 4)))), ("0x801", lambda: append(ints(3, 4), new_lens=ints(2, 1))),
             ("0x802", lambda: append(ints(3, 64))), ("0x803", lambda: wrong_page(lambda: append(ints(3, 4))))]
    for site, wrong in cases + cases[::-1]:
        wrong()
        with pytest.raises(gm.MercuryError, match=site) as e:
            gm.mercury_sync_status()
        assert e.value.status == gm.MERCURY_EBOUNDS
        gm.mercury_sync_status()


# -------------------------------------------------------------------------------- captures

FIRST_CAPTURE = """
import sys
import torch
from long_context_sharded_gb300 import mercury as m
torch.manual_seed(0)
k, v = (torch.randn(300, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
q, x = torch.randn(2, 4, 1, 64, device="cuda").bfloat16(), torch.randn(2, 2, 1, 64, device="cuda").bfloat16()
short, long = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([5, 7], [2000, 2300]))
out, lse, rot = torch.zeros(2, 4, 1, 64, device="cuda"), torch.zeros(2, 4, 1, device="cuda"), torch.zeros_like(q)
cache, plan = m.PagedCache(k, v, table), m.mercury_rope_init(64)
# the only call before: lengths for which nothing is split
m.mercury_attn_paged(q, m.PagedCache(k, v, table[:, :2].contiguous()), short, out=out, lse=lse)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    m.mercury_rope(q, plan, start=3, out=rot)
    m.mercury_kv_append(cache, x, x, short, rope=plan)
    m.mercury_attn_paged(q, cache, long, out=out, lse=lse)
g.replay()
m.mercury_sync_status()
got = [t.clone() for t in (out, lse, rot)]
m.mercury_rope(q, plan, start=3, out=rot)
m.mercury_attn_paged(q, cache, long, out=out, lse=lse)
m.mercury_sync_status()
assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, rot)))
"""


@pytest.mark.gpu
def test_a_call_that_split_nothing_prepares_for_one_that_does(gm):
    """In a process of its own: after one uncaptured call of a shape class any other of it can be captured."""
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------- what the header says

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Sq", [(2, 1), (8, 1), (32, 1), (16, 4)])
def test_infinite_values_that_every_row_sees(gm, d, Hq, Sq):
    """Their columns are not finite in the rows of their head, for single tokens and drafted ones; all else is right."""
    n, page, Hkv, B = 700, 16, 2, 3
    gen = torch.Generator("cuda").manual_seed(d + Hq)
    k_cache, v_cache, table, _ = make_cache(B, Hkv, d, page, -(-n // page), BF16, gen)
    for i, value in enumerate((math.inf, -math.inf, math.nan)):
        v_cache[table[i, 7].long(), 1, 5, i + 3] = value
    q = torch.randn(B, Hq, Sq, d, generator=gen, device="cuda").to(BF16)
    out, lse = gm.mercury_attn_paged(q, gm.PagedCache(k_cache, v_cache, table),
                                     torch.full((B,), n, dtype=torch.int32, device="cuda"))
    gm.mercury_sync_status()
    hit = torch.zeros_like(out, dtype=torch.bool)
    for i in range(B):
        hit[i, Hq // Hkv:, :, i + 3] = True
    assert torch.equal(~torch.isfinite(out), hit)
    for b in range(B):
        k, v = gather_states(k_cache, None, table[b], n), gather_states(v_cache, None, table[b], n)
        o, l, eo, el = attention(q[b], k, torch.where(torch.isfinite(v), v, 0.0), [n - Sq + i + 1 for i in range(Sq)])
        assert_within(out[b][~hit[b]], o[~hit[b]], eo[~hit[b]], "O")
        assert_within(lse[b], l, el, "LSE")


@pytest.mark.gpu
def test_append_rounds_to_even_in_8_bits(gm):
    """300 is nearer to 288 than to 320, 304 lies between them and goes to the even one, 320."""
    k_cache, v_cache, table, _ = make_cache(1, 1, 64, 4, 1, E4M3, torch.Generator("cuda").manual_seed(0))
    one = torch.ones(1, device="cuda")
    k = torch.zeros(1, 1, 1, 64, dtype=BF16, device="cuda")
    x = [1e5, -1e5, math.inf, -math.inf, 300.0, 304.0, -304.0, 272.0, 1e-3, 2.0 ** -10, -2.0 ** -10, 3 * 2.0 ** -10]
    k[..., :len(x)] = torch.tensor(x, device="cuda").to(BF16)
    k[..., 63] = math.nan
    gm.mercury_kv_append(gm.PagedCache(k_cache, v_cache, table, k_scale=one, v_scale=one), k, k,
                         torch.zeros(1, dtype=torch.int32, device="cuda"))
    gm.mercury_sync_status()
    for c in (k_cache, v_cache):
        row = c.view(torch.uint8)[table[0, 0].long(), 0, 0].view(E4M3).float().tolist()
        assert row[:len(x)] == [448.0, -448.0, 448.0, -448.0, 288.0, 320.0, -320.0, 256.0, 2.0 ** -9, 0.0, 0.0, 2.0 ** -8]
        assert math.isnan(row[63])


@pytest.mark.gpu
def test_inputs_are_left_as_they_were(gm):
    gen = torch.Generator("cuda").manual_seed(2)
    k_cache, v_cache, table, _ = make_cache(2, 2, 64, 16, 4, BF16, gen)
    cache, plan = gm.PagedCache(k_cache, v_cache, table), gm.mercury_rope_init(64)
    q, k, v = (torch.randn(2, h, 3, 64, generator=gen, device="cuda").to(BF16) for h in (4, 2, 2))
    past, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([3, 20], [[5, 6, 7], [8, 9, 10]]))
    total = past + 3
    inputs = (q, k, v, past, pos, total, table)
    before = [t.clone() for t in inputs]
    rot = gm.mercury_kv_append(cache, k, v, past, rope=plan, q=q)
    stored = k_cache.clone(), v_cache.clone()
    gm.mercury_rope(q, plan, pos, inverse=True)
    gm.mercury_attn_paged(rot, cache, total)
    gm.mercury_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(inputs, before))
    assert torch.equal(k_cache, stored[0]) and torch.equal(v_cache, stored[1])


def test_a_table_of_too_many_tiles_is_refused(m):
    P = 0x100000
    c = cache_struct(m, max_pages=1 << 26, table_stride=1 << 26, B=40)
    assert m.lib.mercury_attn_paged(P, None, ctypes.byref(c), P, None, 40, 4, 1, 1, P, P, None) == m.MERCURY_EINVAL
    assert b"tiles" in m.lib.mercury_last_error()
