"""The operators that make a long context's cache smaller, as measured cases.

In serving, the cache is what a long context costs: in memory, and, since every new token reads all of it, in time.
Four operators that a serving loop runs together hold it down:

* ``append`` -- new keys and values into a paged cache of 4 bits (e2m1 elements, an e4m3 scale for every 16 of a head
                and a 32-bit one for the head), the keys rotated on the way and the queries of the same tokens with
                them, and the whole context read back as 16-bit keys and values, as the attention of a prompt's chunk
                takes them;
* ``attn``   -- attention of one new token (or a few drafted ones) over that cache, O and the log-sum-exp;
* ``mass``   -- the attention weight that each cached key got from those tokens, added to what it had;
* ``evict``  -- the keys and values with the most of it, and the first and last ones, into a shorter cache.

``run`` computes an operator in its plain form, or, where ``own`` is true, by the library's own calls.  Where a
batch is ragged its lengths are spread evenly between the case's bounds and only their order goes by the seed, so
that the work of a case is known without its inputs.
"""
import math

import numpy as np
import torch

own = False

ROPE_BASE = 500000.0
BLOCK = 16  # elements of a head that share a scale
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of e2m1's codes without their sign
BYTES = {"bf16": 2.0, "e4m3": 1.0, "e2m1": 0.5 + 1.0 / BLOCK}  # of a cached element


# ----------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of 32 sequences, short contexts
        dict(name="append_token_b32", op="append", B=32, Hq=32, Hkv=8, S=1, d=128, page=16, rot=128, interleaved=False,
             past_lo=1, past_hi=127),
        # the last 8K chunk of a 32K prompt: the chunk's attention takes the whole context
        dict(name="append_chunk_8k_of_32k", op="append", B=1, Hq=32, Hkv=8, S=8192, d=128, page=64, rot=128,
             interleaved=False, past_lo=24576, past_hi=24576),
        # a padded batch of prompts behind cached ones, part of a small head rotated, interleaved pairs
        dict(name="append_ragged_d64", op="append", B=6, Hq=16, Hkv=4, S=1000, d=64, page=32, rot=32, interleaved=True,
             past_lo=0, past_hi=777),
        # one token of one sequence behind a 4K context: latency
        dict(name="attn_b1_4k", op="attn", B=1, Hq=32, Hkv=8, Sq=1, d=128, page=16, len_lo=4096, len_hi=4096,
             bf16_out=False),
        # one token of one sequence behind the 128K context of the headline model configuration
        dict(name="attn_b1_128k", op="attn", B=1, Hq=64, Hkv=8, Sq=1, d=128, page=64, len_lo=131072, len_hi=131072,
             bf16_out=True),
        # a serving batch with short and long contexts
        dict(name="attn_b16_ragged_32k", op="attn", B=16, Hq=32, Hkv=8, Sq=1, d=128, page=64, len_lo=700, len_hi=32768,
             bf16_out=False),
        # four drafted tokens to be verified, fewer in some sequences, small heads
        dict(name="attn_b8_draft4_d64", op="attn", B=8, Hq=32, Hkv=8, Sq=4, d=64, page=16, len_lo=900, len_hi=8191,
             bf16_out=False),
        # a decode step's weights, kept at every step
        dict(name="mass_token_b8_32k", op="mass", B=8, Hq=32, Hkv=8, Sq=1, d=128, page=64, elem="bf16", len_lo=20000,
             len_hi=32768, add=True),
        # the weights that a prompt's last 32 tokens give, from a 4-bit cache, once before keys are dropped
        dict(name="mass_window32_16k_e2m1", op="mass", B=2, Hq=32, Hkv=8, Sq=32, d=128, page=32, elem="e2m1",
             len_lo=9000, len_hi=16384, add=False),
        # a few drafted tokens over a small 8-bit cache: latency
        dict(name="mass_draft3_2k_e4m3", op="mass", B=2, Hq=16, Hkv=4, Sq=3, d=64, page=16, elem="e4m3", len_lo=700,
             len_hi=2047, add=True),
        # a 32K context down to 4K
        dict(name="evict_b1_32k_to_4k", op="evict", B=1, Hkv=8, d=128, page=64, elem="bf16", len_lo=32768, len_hi=32768,
             keep=4096, first=4, last=512),
        # a batch, some sequences already short enough, 8-bit
        dict(name="evict_b16_ragged_e4m3", op="evict", B=16, Hkv=8, d=128, page=32, elem="e4m3", len_lo=500, len_hi=16000,
             keep=2048, first=4, last=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most = {k: max(most.get(k, 0), v) for k, v in w.items()}
    while True:
        c = _drawn(rng)
        w = work(c)
        wide = c["B"] * c.get("Hq", 1) * c.get("Sq", 1) * c.get("len_hi", 1) if c["op"] in ("attn", "mass") else 0
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and wide <= 1 << 30:
            return c


def _drawn(rng):
    op = rng.choice(["append", "attn", "attn", "mass", "evict"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 5])
    page = rng.choice([8, 16, 16, 32, 64, 128, 24])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    if op == "append":
        lo = _log(rng, 1, 8000) - 1
        return dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, S=_log(rng, 1, 16384), d=d, page=page,
                    rot=rng.choice([d, d, d // 2, 24]), interleaved=rng.random() < 0.5, past_lo=lo,
                    past_hi=lo + rng.randint(0, 500))
    elem = rng.choice(["bf16", "e4m3", "e2m1"])
    if op == "evict":
        hi = _log(rng, 64, 131072)
        first, last = rng.randint(0, 8), _log(rng, 1, 512) - 1
        return dict(op=op, B=_log(rng, 1, 32), Hkv=Hkv, d=d, page=page, elem=rng.choice(["bf16", "e4m3"]),
                    len_lo=rng.randint(1, hi), len_hi=hi, keep=max(first + last, _log(rng, 16, hi)), first=first, last=last)
    Sq = rng.choice([1, 1, 1, 2, 3, 4, 7] if op == "attn" else [1, 1, 4, 7, 16, 33, 64])
    hi = max(_log(rng, 1, 131072), Sq)
    c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, Sq=Sq, d=d, page=page, len_lo=rng.randint(Sq, hi), len_hi=hi)
    return c | (dict(bf16_out=rng.random() < 0.5) if op == "attn" else dict(elem=elem, add=rng.random() < 0.5))


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) if n > 1 else hi for i in range(n)]


def _new_lens(c, S):
    """New tokens of each sequence: a padded batch where there is more than one of each."""
    return _spread(1, S, c["B"] - 1) + [S] if c["B"] > 1 and S > 1 else [S] * c["B"]


def work(case):
    c = case
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "append":
        new, e = sum(_new_lens(c, c["S"])), BYTES["e2m1"]
        all_of = sum(_spread(c["past_lo"], c["past_hi"], B)) + new
        return {"bytes": int(new * d * (2 * Hkv * (2 + e) + 4 * c["Hq"]) + all_of * d * 2 * Hkv * (e + 2)),
                "flops": 3 * new * c["rot"] * (c["Hq"] + Hkv)}
    lens = _spread(c["len_lo"], c["len_hi"], B)
    if c["op"] == "attn":
        rows = B * c["Hq"] * c["Sq"]
        return {"bytes": int(2 * sum(lens) * Hkv * d * BYTES["e2m1"] + rows * (d * (2 + (2 if c["bf16_out"] else 4)) + 4)),
                "flops": 4 * d * c["Hq"] * c["Sq"] * sum(lens)}
    if c["op"] == "mass":
        return {"bytes": int(sum(lens) * Hkv * (d * BYTES[c["elem"]] + (8 if c["add"] else 4)) +
                             B * c["Hq"] * c["Sq"] * (2 * d + 4)),
                "flops": 2 * d * c["Hq"] * c["Sq"] * sum(lens)}
    kept = sum(min(n, c["keep"]) for n in lens)
    return {"bytes": int(sum(lens) * Hkv * 4 + kept * Hkv * (4 * d * BYTES[c["elem"]] + 8)), "flops": sum(lens) * Hkv}


# ---------------------------------------------------------------------------------------------------- the inputs

def _frequencies(rot):
    return ROPE_BASE ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)


def _packed(codes, scales):
    """Rows of d codes (0 to 15) and their d/16 scales' bytes as rows of the cache: two codes a byte, the first in the
    lower half, then the scales."""
    return torch.cat((codes[..., 0::2] | codes[..., 1::2] << 4, scales), dim=-1)


def _like_states(shape, gen):
    """A 4-bit cache's rows, of normal values."""
    x = torch.randn(shape, generator=gen, device="cuda").unflatten(-1, (-1, BLOCK))
    s = (x.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    codes = torch.bucketize(x.abs() / s.float(), borders).to(torch.uint8) | (x < 0).to(torch.uint8) << 3
    return _packed(codes.flatten(-2), s.view(torch.uint8).squeeze(-1))


def _pages(c, totals, gen, elem, spare=3):
    """A cache whose pages lie in no order, the table of them (-1 where a sequence has no page), and the scales."""
    P, B, d = c["page"], c["B"], c["d"]
    used = [-(-t // P) for t in totals]
    n = sum(used) + spare
    caches = []
    for _ in range(2):
        kind = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[elem]
        x = torch.empty((n, c["Hkv"], P, d // 2 + d // BLOCK if elem == "e2m1" else d), dtype=kind, device="cuda")
        for part in x.split(max(1, (1 << 27) // (c["Hkv"] * P * d))):
            shape = part.shape[:3] + (d,)
            part.copy_(_like_states(shape, gen) if elem == "e2m1" else
                       torch.randn(shape, generator=gen, device="cuda") * (40.0 if elem == "e4m3" else 1.0))
        caches.append(x)
    order = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    scales = [None, None]
    if elem != "bf16":
        lo, more = (0.02, 0.01) if elem == "e4m3" else (0.8, 0.4)
        scales = [torch.rand(c["Hkv"], generator=gen, device="cuda") * more + lo for _ in range(2)]
    return caches, table, scales


def _shuffled(values, gen):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=gen, device="cuda")]


def prepare(case, seed):
    c = case
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    gen = torch.Generator("cuda").manual_seed(seed)
    if c["op"] == "append":
        order = torch.randperm(B, generator=gen, device="cuda")
        past = torch.tensor(_spread(c["past_lo"], c["past_hi"], B), dtype=torch.int32, device="cuda")[order]
        new = torch.tensor(_new_lens(c, c["S"]), dtype=torch.int32, device="cuda")[order]
        caches, table, scales = _pages(c, (past + new).tolist(), gen, "e2m1")
        qkv = torch.randn(B, c["S"], c["Hq"] + 2 * Hkv, d, generator=gen, device="cuda").bfloat16().transpose(1, 2)
        q, k, v = qkv.split([c["Hq"], Hkv, Hkv], dim=1)
        read = [torch.zeros(B, Hkv, int((past + new).max()), d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        s = dict(c=c, elem="e2m1", q=q, k=k, v=v, past=past, new=new, lens=past + new, caches=caches, table=table,
                 scales=scales, q_out=torch.zeros(B, c["Hq"], c["S"], d, dtype=torch.bfloat16, device="cuda"), read=read,
                 freq=_frequencies(c["rot"]))
        if own:
            from long_context_sharded_gb300 import mercury as m
            s["plan"] = m.mercury_rope_init(c["rot"], base=ROPE_BASE, interleaved=c["interleaved"])
    else:
        lens = _shuffled(_spread(c["len_lo"], c["len_hi"], B), gen)
        elem = "e2m1" if c["op"] == "attn" else c["elem"]
        caches, table, scales = _pages(c, lens.tolist(), gen, elem)
        s = dict(c=c, elem=elem, lens=lens, caches=caches, table=table, scales=scales)
    if c["op"] in ("attn", "mass"):
        s["q"] = torch.randn(B, c["Hq"], c["Sq"], d, generator=gen, device="cuda").mul_(2.0).bfloat16()
        s["new"] = torch.tensor(_new_lens(c, c["Sq"]), dtype=torch.int32, device="cuda")
        s["lse"] = torch.zeros(s["q"].shape[:3], device="cuda")
    if c["op"] == "attn":
        s["out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16 if c["bf16_out"] else torch.float32, device="cuda")
    if c["op"] == "mass":
        s["lse"].copy_(_attention(s, weights=False)[1])
        s["mass"] = torch.rand(B, Hkv, int(lens.max()), generator=gen, device="cuda") if c["add"] else None
        s["sums"] = torch.zeros(B, Hkv, int(lens.max()), device="cuda")
    if c["op"] == "evict":
        # few keys with much, many with little, the newest with none
        s["mass"] = torch.exp(2.0 * torch.randn(B, Hkv, int(lens.max()), generator=gen, device="cuda") - 2.0)
        s["mass"] *= torch.rand(s["mass"].shape, generator=gen, device="cuda") < 0.97
        into, s["into_table"], _ = _pages(c, [min(n, c["keep"]) for n in lens.tolist()], gen, elem)
        s["into"] = into
        s["kept"] = torch.full((B, Hkv, c["keep"]), -1, dtype=torch.int32, device="cuda")
        s["kept_mass"] = torch.zeros(B, Hkv, c["keep"], device="cuda")
        s["kept_lens"] = torch.zeros_like(lens)
    if own:
        from long_context_sharded_gb300 import mercury as m
        s["cache"] = m.PagedCache(caches[0], caches[1], table, k_scale=scales[0], v_scale=scales[1])
        if c["op"] == "evict":
            s["into_cache"] = m.PagedCache(s["into"][0], s["into"][1], s["into_table"], k_scale=scales[0], v_scale=scales[1])
    return s


# --------------------------------------------------------------------------------------------------- the operators

def _turned(x, pos, freq, c):
    """x [B,H,S,d] in 64 bits with its first c["rot"] elements turned by pos [B,S] times the frequencies."""
    angle = pos.double()[:, None, :, None] * torch.from_numpy(freq).to(pos.device)
    cos, sin = angle.cos(), angle.sin()
    x, rot = x.double(), c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _quantized(x, scale):
    """x [tokens, heads, d] in 64 bits as rows of a 4-bit cache, scale [heads]: each block's scale is the e4m3 nearest
    to its largest magnitude over 6 scale[head], each code the e2m1 nearest to the element over both scales, ties to
    even.  In 64 bits throughout, where a quotient of such inputs is never taken for a tie."""
    x = x.unflatten(-1, (-1, BLOCK))
    g = scale.double()[:, None, None]
    want = x.abs().amax(-1, keepdim=True) / (6.0 * g)
    step = torch.exp2(torch.frexp(want)[1].double().clamp(min=-5.0) - 4.0)  # e4m3: four bits, down to 2^-9
    s = (torch.round(want / step) * step).clamp(max=448.0)
    m = torch.where(s > 0, x.abs() / torch.where(s > 0, s * g, 1.0), 0.0)
    code = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte() + (m > 2.5).byte() +
            (m >= 3.5).byte() + (m > 5.0).byte())
    code |= (x < 0).byte() << 3
    return _packed(code.flatten(-2), s.squeeze(-1).float().to(torch.float8_e4m3fn).view(torch.uint8))


def _values(rows, elem, d):
    """Cached rows [..., bytes] as 32-bit numbers, without their head's scale."""
    if elem != "e2m1":
        return rows.float()
    codes = torch.stack((rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4), dim=-1).flatten(-2).long()
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=rows.device)
    scales = rows[..., d // 2:].contiguous().view(torch.float8_e4m3fn).float()
    return (table[codes].unflatten(-1, (-1, BLOCK)) * scales[..., None]).flatten(-2)


def _states(s, i):
    """Keys (0) or values (1) of every sequence, [B,Hkv,n,d] in 32 bits; n is a whole number of pages."""
    c, cache = s["c"], s["caches"][i]
    pages = s["table"].clamp(min=0).long()
    rows = cache.view(torch.uint8)[pages].view(cache.dtype) if s["elem"] == "e4m3" else cache[pages]
    x = _values(rows.transpose(1, 2).flatten(2, 3), s["elem"], c["d"])
    return x if s["scales"][i] is None else x.mul_(s["scales"][i][:, None, None])


def _attention(s, weights):
    """Scores [B,Hkv,G,Sq,n] of the new tokens and their log-sum-exp [B,Hq,Sq], or O [B,Hkv,G,Sq,d] and it."""
    c = s["c"]
    B, Hkv, Sq, d = c["B"], c["Hkv"], c["Sq"], c["d"]
    G = c["Hq"] // Hkv
    q = s["q"].float().reshape(B, Hkv, G * Sq, d) / math.sqrt(d)
    scores = (q @ _states(s, 0).transpose(2, 3)).reshape(B, Hkv, G, Sq, -1)
    step = torch.arange(Sq, device="cuda")
    last = (s["lens"] - s["new"])[:, None] + step  # the last key that each new token sees
    key = torch.arange(scores.shape[-1], device="cuda")
    seen = (key <= last[..., None]) & (key < s["lens"][:, None, None])
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = (scores - top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).reshape(B, -1, Sq)
    if not weights:
        return scores, lse
    return (p.reshape(B, Hkv, G * Sq, -1) @ _states(s, 1)).reshape(B, Hkv, G, Sq, d) / total, lse


def _plain_append(s):
    c = s["c"]
    step = torch.arange(c["S"], device="cuda")
    pos = s["past"][:, None].long() + step
    live = step < s["new"][:, None]
    q = _turned(s["q"], pos, s["freq"], c).bfloat16()
    s["q_out"].copy_(torch.where(live[:, None, :, None], q, s["q_out"]))
    page = s["table"].gather(1, torch.where(live, pos // c["page"], 0)).long()[live]
    row = (pos % c["page"])[live]
    for cache, x, scale in zip(s["caches"], (_turned(s["k"], pos, s["freq"], c), s["v"].double()), s["scales"]):
        cache[page, :, row] = _quantized(x.transpose(1, 2)[live], scale)
    live = torch.arange(s["read"][0].shape[2], device="cuda") < s["lens"][:, None]
    for i in range(2):
        x = _states(s, i)[:, :, :live.shape[1]]
        s["read"][i].copy_(torch.where(live[:, None, :, None], x.bfloat16(), s["read"][i]))
    return {"q": s["q_out"], "k": s["read"][0], "v": s["read"][1]}


def _plain_attn(s):
    c = s["c"]
    out, lse = _attention(s, weights=True)
    live = (torch.arange(c["Sq"], device="cuda") < s["new"][:, None])[:, None]
    s["out"].copy_(torch.where(live[..., None], out.reshape(s["out"].shape).to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(live, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_mass(s):
    c = s["c"]
    scores, _ = _attention(s, weights=False)
    p = (scores - s["lse"].reshape(scores.shape[:4])[..., None]).exp_()
    p.mul_((torch.arange(c["Sq"], device="cuda") < s["new"][:, None])[:, None, None, :, None])
    width = s["sums"].shape[2]
    got = p.sum((2, 3))[..., :width]
    if s["mass"] is not None:
        got = got + s["mass"]
    live = torch.arange(width, device="cuda") < s["lens"][:, None, None]
    return s["sums"].copy_(torch.where(live, got, s["sums"]))


def _plain_evict(s):
    c = s["c"]
    P, lens = c["page"], s["lens"][:, None, None].long()
    at = torch.arange(s["mass"].shape[2], device="cuda")
    want = s["mass"].masked_fill((at < c["first"]) | (at >= lens - c["last"]), float("inf"))
    want = want.masked_fill(at >= lens, float("-inf"))
    # by weight, the earlier of two equal ones first
    order = torch.sort(want, dim=-1, descending=True, stable=True)[1]
    kept = torch.zeros_like(want, dtype=torch.bool).scatter_(2, order, (at < lens.clamp(max=c["keep"])).expand_as(order))
    b, h, src = kept.nonzero(as_tuple=True)  # in order of position
    slot = (kept.cumsum(-1) - 1)[b, h, src]
    s["kept"][b, h, slot] = src.int()
    s["kept_mass"][b, h, slot] = s["mass"][b, h, src]
    s["kept_lens"].copy_(s["lens"].clamp(max=c["keep"]))
    here = s["table"][b, src // P].long(), h, src % P
    there = s["into_table"][b, slot // P].long(), h, slot % P
    for a, z in zip(s["caches"], s["into"]):
        z.view(torch.uint8)[there] = a.view(torch.uint8)[here]
    return {"lens": s["kept_lens"], "kept": s["kept"], "mass": s["kept_mass"], "k": s["into"][0], "v": s["into"][1]}


def run(state):
    s = state
    c = s["c"]
    if own:
        from long_context_sharded_gb300 import mercury as m
        if c["op"] == "append":
            m.mercury_kv_append(s["cache"], s["k"], s["v"], s["past"], new_lens=s["new"], rope=s["plan"], q=s["q"],
                                q_out=s["q_out"])
            m.mercury_kv_read(s["cache"], s["lens"], k_out=s["read"][0], v_out=s["read"][1])
            return {"q": s["q_out"], "k": s["read"][0], "v": s["read"][1]}
        if c["op"] == "attn":
            call = m.mercury_attn_paged_bf16 if c["bf16_out"] else m.mercury_attn_paged
            call(s["q"], s["cache"], s["lens"], new_lens=s["new"], causal=True, out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if c["op"] == "mass":
            return m.mercury_attn_paged_mass(s["q"], s["cache"], s["lens"], s["lse"], new_lens=s["new"], causal=True,
                                             mass=s["mass"], out=s["sums"])
        m.mercury_kv_evict(s["cache"], s["into_cache"], s["mass"], s["lens"], c["keep"], first=c["first"], last=c["last"],
                           out_lens=s["kept_lens"], kept=s["kept"], out_mass=s["kept_mass"])
        return {"lens": s["kept_lens"], "kept": s["kept"], "mass": s["kept_mass"], "k": s["into"][0], "v": s["into"][1]}
    return {"append": _plain_append, "attn": _plain_attn, "mass": _plain_mass, "evict": _plain_evict}[c["op"]](s)


# ------------------------------------------------------------------------------------- the definitions in 64 bits

def _nearest(x, values):
    """The index of the value nearest to each of x, of two equally near ones the even one."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    above = torch.searchsorted(v, x).clamp(1, len(values) - 1)
    below = above - 1
    up, down = v[above] - x, x - v[below]
    return torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)


def _held(x, scale):
    """What a 4-bit cache holds of x [n, d] with its head's scale."""
    scales = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    blocks = x.reshape(-1, BLOCK)
    s = torch.tensor(scales, dtype=torch.float64, device=x.device)[
        _nearest(blocks.abs().max(1).values / (6.0 * scale), scales)].unsqueeze(1)
    sized = torch.where(s == 0, torch.zeros_like(blocks), blocks.abs() / (s * scale).clamp(min=1e-300))
    held = torch.tensor(VALUES, dtype=torch.float64, device=x.device)[_nearest(sized, VALUES)]
    return (torch.copysign(held, blocks) * s * scale).reshape(x.shape)


def _unpacked(rows, elem, d, scale):
    """Cached rows of one head [n, bytes] in 64 bits."""
    if elem == "bf16":
        return rows.double()
    if elem == "e4m3":
        return rows.double() * scale.double()
    out = torch.empty(rows.shape[0], d, dtype=torch.float64, device=rows.device)
    v = torch.tensor(VALUES, dtype=torch.float64, device=rows.device)
    for at in (0, 1):
        code = (rows[:, :d // 2] >> (4 * at) & 15).long()
        out[:, at::2] = v[code % 8] * (1 - 2 * (code // 8))
    s = rows[:, d // 2:].contiguous().view(torch.float8_e4m3fn).double()
    return out * s.repeat_interleave(BLOCK, dim=1) * scale.double()


def _head(s, i, b, h, n):
    """The first n keys (0) or values (1) of a head of a sequence, in 64 bits."""
    at = torch.arange(n, device="cuda")
    page, row = s["table"][b].long()[torch.div(at, s["c"]["page"], rounding_mode="floor")], at % s["c"]["page"]
    cache = s["caches"][i]
    rows = cache.view(torch.uint8)[page, h, row].view(cache.dtype) if s["elem"] == "e4m3" else cache[page, h, row]
    return _unpacked(rows, s["elem"], s["c"]["d"], None if s["scales"][i] is None else s["scales"][i][h])


def _turned64(x, at, c):
    """x [n, d] at positions [n], turned as complex numbers."""
    y, rot = x.double().clone(), c["rot"]
    rates = torch.tensor([math.exp(-2.0 * i / rot * math.log(ROPE_BASE)) for i in range(rot // 2)], dtype=torch.float64,
                         device=x.device)
    one = torch.arange(0, rot, 2, device=x.device) if c["interleaved"] else torch.arange(rot // 2, device=x.device)
    two = one + (1 if c["interleaved"] else rot // 2)
    angle = at.double().unsqueeze(1) * rates
    z = torch.complex(y[:, one], y[:, two]) * torch.polar(torch.ones_like(angle), angle)
    y[:, one], y[:, two] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    B, Hkv = c["B"], c["Hkv"]
    lens = s["lens"].tolist()
    if c["op"] == "append":
        q, k, v = s["q_out"].double(), s["read"][0].double(), s["read"][1].double()
        past, new = s["past"].tolist(), s["new"].tolist()
        for b in range(B):
            n = new[b]
            at = torch.arange(past[b], past[b] + n, device="cuda")
            for h in range(c["Hq"]):
                q[b, h, :n] = _turned64(s["q"][b, h, :n], at, c)
            for h in range(Hkv):
                k[b, h, :lens[b]] = _head(s, 0, b, h, lens[b])
                v[b, h, :lens[b]] = _head(s, 1, b, h, lens[b])
                k[b, h, past[b]:lens[b]] = _held(_turned64(s["k"][b, h, :n], at, c), s["scales"][0][h].double())
                v[b, h, past[b]:lens[b]] = _held(s["v"][b, h, :n].double(), s["scales"][1][h].double())
        return {"q": q, "k": k, "v": v}
    if c["op"] == "evict":
        kept, mass = s["kept"].clone(), s["kept_mass"].double()
        for b in range(B):
            n, m = lens[b], min(lens[b], c["keep"])
            for h in range(Hkv):
                free = torch.arange(n, device="cuda")
                sure = (free < c["first"]) | (free >= n - c["last"])
                if n > m:
                    rest = free[~sure]
                    best = torch.argsort(-s["mass"][b, h, rest].double(), stable=True)[:m - int(sure.sum())]
                    free = torch.cat((free[sure], rest[best])).sort().values
                kept[b, h, :m] = free.int()
                mass[b, h, :m] = s["mass"][b, h, free].double()
        return {"lens": s["lens"].clamp(max=c["keep"]), "kept": kept, "mass": mass, "k": None, "v": None}
    new, G = s["new"].tolist(), c["Hq"] // Hkv
    if c["op"] == "attn":
        out, lse = s["out"].double(), s["lse"].double()
    else:
        sums = s["sums"].double()
    for b in range(B):
        for h in range(Hkv):
            k = _head(s, 0, b, h, lens[b])
            if c["op"] == "attn":
                v = _head(s, 1, b, h, lens[b])
            else:
                sums[b, h, :lens[b]] = 0.0 if s["mass"] is None else s["mass"][b, h, :lens[b]].double()
            x = s["q"][b, h * G:(h + 1) * G, :new[b]].double() @ k.T / math.sqrt(c["d"])
            past = torch.arange(new[b], device="cuda") + lens[b] - new[b]
            x = torch.where(torch.arange(lens[b], device="cuda") <= past.unsqueeze(1), x, -math.inf)
            if c["op"] == "attn":
                lse[b, h * G:(h + 1) * G, :new[b]] = torch.logsumexp(x, 2)
                out[b, h * G:(h + 1) * G, :new[b]] = torch.softmax(x, 2) @ v
            else:
                p = torch.exp(x - s["lse"][b, h * G:(h + 1) * G, :new[b]].double().unsqueeze(2))
                sums[b, h, :lens[b]] += p.sum((0, 1))
    return {"out": out, "lse": lse} if c["op"] == "attn" else sums
