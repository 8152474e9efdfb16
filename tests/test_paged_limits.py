"""The serving operators where their promises are hardest to keep: outputs that a call makes for another stream,
values that are not finite beside one another, sums over long contexts, weights far below the largest, copies that
never come.

Bounds are derived where they are used; a rounding is off by at most half a step, as in test_paged.py, whose 64-bit
definitions these tests share.
"""
import contextlib
import types

import pytest
import torch

from tests.test_paged import BF16, FP32, cache_struct, gm, m, make_cache  # noqa: F401  (gm, m: fixtures)


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
