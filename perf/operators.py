"""The serving-side operators of the library, as measured cases.

Three operators that a serving loop over a long context runs together:

* ``rope``   -- rotary positions of a prompt's (or one token's) heads, half and interleaved pairs, a part of the
                head or all of it, frequencies as they are or scaled for a longer context, and the transposed
                rotation that carries gradients back;
* ``append`` -- new keys and values into a paged cache (bf16, or e4m3 with one scale per head), the keys rotated on
                the way and the queries of the same tokens with them;
* ``attn``   -- attention of one new token (or a few drafted ones) over that cache, O and the log-sum-exp.

``run`` computes an operator in its plain form, or, where ``own`` is true, by the library's own calls.  Where a
batch is ragged its lengths are spread evenly between the case's bounds and only their order goes by the seed, so
that the work of a case is known without its inputs.
"""
import math

import numpy as np
import torch

own = False

ROPE_BASE = 500000.0
ROPE_ORIGINAL = 8192


# ----------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step's query and key heads of a batch of 8 (Hq 32, Hkv 8), far positions
        dict(name="rope_token_b8_h40", op="rope", B=8, H=40, S=1, d=128, rot=128, interleaved=False, scaling="none",
             start=131000, inverse=False, fp32=False, fused=True),
        # the query and key heads of a 32K prompt, straight from a fused projection, frequencies scaled for its length
        dict(name="rope_prompt_32k_h40_scaled", op="rope", B=1, H=40, S=32768, d=128, rot=128, interleaved=False,
             scaling="yarn", start=0, inverse=False, fp32=False, fused=True),
        # the gradient of a half-rotated head with interleaved pairs, an odd length, 32-bit
        dict(name="rope_gradient_interleaved_part", op="rope", B=2, H=12, S=4099, d=64, rot=32, interleaved=True,
             scaling="linear", start=17, inverse=True, fp32=True, fused=False),
        # one decode step of 32 sequences
        dict(name="append_token_b32", op="append", B=32, Hq=32, Hkv=8, S=1, d=128, page=16, e4m3=False, rot=128,
             interleaved=False, past_lo=1, past_hi=127),
        # a 32K prompt into an empty cache
        dict(name="append_prompt_32k", op="append", B=1, Hq=32, Hkv=8, S=32768, d=128, page=64, e4m3=False, rot=128,
             interleaved=False, past_lo=0, past_hi=0),
        # a padded batch of prompts behind cached ones, into an 8-bit cache, part of the head rotated
        dict(name="append_ragged_e4m3", op="append", B=6, Hq=16, Hkv=4, S=1000, d=64, page=32, e4m3=True, rot=32,
             interleaved=True, past_lo=0, past_hi=777),
        # one token of one sequence behind a 4K context: latency
        dict(name="attn_b1_4k", op="attn", B=1, Hq=32, Hkv=8, Sq=1, d=128, page=16, e4m3=False, len_lo=4096,
             len_hi=4096, bf16_out=False),
        # one token of one sequence behind the 128K context of the headline model configuration
        dict(name="attn_b1_128k", op="attn", B=1, Hq=64, Hkv=8, Sq=1, d=128, page=64, e4m3=False, len_lo=131072,
             len_hi=131072, bf16_out=True),
        # a serving batch with short and long contexts
        dict(name="attn_b16_ragged_32k", op="attn", B=16, Hq=64, Hkv=8, Sq=1, d=128, page=64, e4m3=False, len_lo=700,
             len_hi=32768, bf16_out=False),
        # many short contexts, one query head per key head
        dict(name="attn_b64_short_mha_d64", op="attn", B=64, Hq=16, Hkv=16, Sq=1, d=64, page=16, e4m3=False, len_lo=1,
             len_hi=2047, bf16_out=True),
        # the 8-bit cache
        dict(name="attn_b8_32k_e4m3", op="attn", B=8, Hq=32, Hkv=8, Sq=1, d=128, page=32, e4m3=True, len_lo=20000,
             len_hi=32768, bf16_out=True),
        # four drafted tokens to be verified, fewer in some sequences
        dict(name="attn_b8_draft4_8k", op="attn", B=8, Hq=32, Hkv=8, Sq=4, d=128, page=16, e4m3=False, len_lo=900,
             len_hi=8191, bf16_out=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        c = _drawn(rng)
        if work(c)["bytes"] <= most:
            return c


def _drawn(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, d // 4, 24])
        return dict(op=op, B=_log(rng, 1, 64), H=rng.randint(1, 72), S=_log(rng, 1, 32768), d=d, rot=rot,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    start=_log(rng, 1, 1000000) - 1, inverse=rng.random() < 0.3, fp32=rng.random() < 0.3,
                    fused=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8, 8, 5])
    page = rng.choice([8, 16, 16, 32, 64, 128, 24])
    e4m3 = rng.random() < 0.35
    if op == "append":
        lo = _log(rng, 1, 8000) - 1
        return dict(op=op, B=_log(rng, 1, 64), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, S=_log(rng, 1, 32768),
                    d=d, page=page, e4m3=e4m3, rot=rng.choice([d, d, d // 2, 24]), interleaved=rng.random() < 0.5,
                    past_lo=lo, past_hi=lo + rng.randint(0, 500))
    hi = _log(rng, 1, 131072)
    Sq = rng.choice([1, 1, 1, 2, 3, 4, 7])
    hi = max(hi, Sq)
    return dict(op=op, B=_log(rng, 1, 64), Hq=Hkv * rng.choice([1, 2, 4, 7, 8, 16]), Hkv=Hkv, Sq=Sq, d=d, page=page,
                e4m3=e4m3, len_lo=rng.randint(Sq, hi), len_hi=hi, bf16_out=rng.random() < 0.5)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) if n > 1 else hi for i in range(n)]


def _new_lens(c, S):
    """New tokens of each sequence: a padded batch where there is more than one of each."""
    return _spread(1, S, c["B"] - 1) + [S] if c["B"] > 1 and S > 1 else [S] * c["B"]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["H"] * c["S"]
        return {"bytes": 2 * n * c["d"] * (4 if c["fp32"] else 2) + 4 * c["B"] * c["S"], "flops": 3 * n * c["rot"]}
    e = 1 if c["e4m3"] else 2
    if c["op"] == "append":
        new = sum(_new_lens(c, c["S"]))
        moved = 2 * c["Hkv"] * (2 + e) + 2 * c["Hq"] * 2
        return {"bytes": new * c["d"] * moved, "flops": 3 * new * c["rot"] * (c["Hq"] + c["Hkv"])}
    lens = _spread(c["len_lo"], c["len_hi"], c["B"])
    rows = c["B"] * c["Hq"] * c["Sq"]
    return {"bytes": 2 * sum(lens) * c["Hkv"] * c["d"] * e + rows * (c["d"] * (2 + (2 if c["bf16_out"] else 4)) + 4),
            "flops": 4 * c["d"] * c["Hq"] * c["Sq"] * sum(lens)}


# ---------------------------------------------------------------------------------------------------- the inputs

def _frequencies(rot, scaling):
    """(radians a position for each pair, factor on the rotated values), by the published formulas."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = ROPE_BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "ntk":
        return (ROPE_BASE * 4.0 ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if scaling == "yarn":
        keep = np.clip((ROPE_ORIGINAL * f / (2 * np.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return keep * f + (1 - keep) * f / 4.0, 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def _plan(rot, interleaved, scaling):
    from long_context_sharded_gb300 import mercury as m
    return m.mercury_rope_init(rot, base=ROPE_BASE, interleaved=interleaved, scaling=scaling, factor=4.0,
                               original_length=ROPE_ORIGINAL)


def _pages(c, totals, gen):
    """A cache whose pages lie in no order, the table of them (-1 where a sequence has no page), and the scales."""
    P, B = c["page"], c["B"]
    used = [-(-t // P) for t in totals]
    n = sum(used) + 3
    shape = (n, c["Hkv"], P, c["d"])
    caches = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.float8_e4m3fn if c["e4m3"] else torch.bfloat16, device="cuda")
        for part in x.split(max(1, (1 << 28) // (c["Hkv"] * P * c["d"]))):
            r = torch.randn(part.shape, generator=gen, device="cuda")
            part.copy_(r * 40.0 if c["e4m3"] else r)
        caches.append(x)
    order = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    scales = [None, None]
    if c["e4m3"]:
        scales = [torch.rand(c["Hkv"], generator=gen, device="cuda") * 0.01 + 0.02 for _ in range(2)]
    return caches, table, scales


def _shuffled(values, gen):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=gen, device="cuda")]


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    if c["op"] == "rope":
        dt = torch.float32 if c["fp32"] else torch.bfloat16
        if c["fused"]:  # heads next to one another for each token, as a projection writes them
            x = torch.randn(c["B"], c["S"], c["H"], c["d"], generator=gen, device="cuda").to(dt).transpose(1, 2)
        else:
            x = torch.randn(c["B"], c["H"], c["S"], c["d"], generator=gen, device="cuda").to(dt)
        first = torch.randint(0, 64, (c["B"], 1), generator=gen, device="cuda") + c["start"]
        pos = (first + torch.arange(c["S"], device="cuda")).to(torch.int32)
        s = dict(c=c, x=x, pos=pos, out=torch.empty_like(x), freq=_frequencies(c["rot"], c["scaling"]))
        if own:
            s["plan"] = _plan(c["rot"], c["interleaved"], c["scaling"])
        return s
    if c["op"] == "append":
        order = torch.randperm(c["B"], generator=gen, device="cuda")
        past = torch.tensor(_spread(c["past_lo"], c["past_hi"], c["B"]), dtype=torch.int32, device="cuda")[order]
        new = torch.tensor(_new_lens(c, c["S"]), dtype=torch.int32, device="cuda")[order]
        caches, table, scales = _pages(c, [a + b for a, b in zip(past.tolist(), new.tolist())], gen)
        heads = c["Hq"] + 2 * c["Hkv"]
        qkv = torch.randn(c["B"], c["S"], heads, c["d"], generator=gen, device="cuda").bfloat16().transpose(1, 2)
        q, k, v = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s = dict(c=c, q=q, k=k, v=v, past=past, new=new, caches=caches, table=table, scales=scales,
                 q_out=torch.zeros(c["B"], c["Hq"], c["S"], c["d"], dtype=torch.bfloat16, device="cuda"),
                 freq=_frequencies(c["rot"], "none"))
        if own:
            s["plan"] = _plan(c["rot"], c["interleaved"], "none")
    else:
        lens = _shuffled(_spread(c["len_lo"], c["len_hi"], c["B"]), gen)
        new = torch.tensor(_new_lens(c, c["Sq"]), dtype=torch.int32, device="cuda")
        caches, table, scales = _pages(c, lens.tolist(), gen)
        q = torch.randn(c["B"], c["Hq"], c["Sq"], c["d"], generator=gen, device="cuda").mul_(2.0).bfloat16()
        s = dict(c=c, q=q, lens=lens, new=new, caches=caches, table=table, scales=scales,
                 out=torch.zeros(q.shape, dtype=torch.bfloat16 if c["bf16_out"] else torch.float32, device="cuda"),
                 lse=torch.zeros(q.shape[:3], device="cuda"))
    if own:
        from long_context_sharded_gb300 import mercury as m
        s["cache"] = m.PagedCache(caches[0], caches[1], table, k_scale=scales[0], v_scale=scales[1])
    return s


# --------------------------------------------------------------------------------------------------- the operators

def _rotated(x, pos, freq, c, inverse=False):
    """x [B,H,S,d] in 32 bits with its first c["rot"] elements turned by pos [B,S] times the frequencies; the angles
    are taken in 64 bits, since a far position leaves 32 no fraction of a turn."""
    f, magnitude = freq
    angle = pos.double()[:, None, :, None] * torch.from_numpy(f).to(pos.device)
    cos, sin = (angle.cos() * magnitude).float(), (angle.sin() * magnitude).float()
    if inverse:
        sin = -sin
    x = x.float()
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _plain_append(s):
    c = s["c"]
    step = torch.arange(c["S"], device="cuda")
    pos = s["past"][:, None].long() + step
    live = step < s["new"][:, None]
    q = _rotated(s["q"], pos, s["freq"], c).bfloat16()
    s["q_out"].copy_(torch.where(live[:, None, :, None], q, s["q_out"]))
    page = s["table"].gather(1, torch.where(live, pos // c["page"], 0)).long()[live]
    row = (pos % c["page"])[live]
    for cache, x, scale in zip(s["caches"], (_rotated(s["k"], pos, s["freq"], c), s["v"].float()), s["scales"]):
        x = x.transpose(1, 2)[live]  # [tokens, heads, d]
        if c["e4m3"]:
            x = (x / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[page, :, row] = x.view(torch.uint8)
        else:
            cache[page, :, row] = x.bfloat16()
    return {"q": s["q_out"], "k_cache": s["caches"][0], "v_cache": s["caches"][1]}


def _plain_attn(s):
    c = s["c"]
    B, Hkv, Sq, d = c["B"], c["Hkv"], c["Sq"], c["d"]
    G = c["Hq"] // Hkv
    pages = s["table"].clamp(min=0).long()

    def states(cache, scale):
        x = cache.view(torch.uint8)[pages].view(cache.dtype) if c["e4m3"] else cache[pages]
        x = x.transpose(1, 2).reshape(B, Hkv, -1, d).float()
        return x if scale is None else x.mul_(scale[:, None, None])

    q = s["q"].float().reshape(B, Hkv, G * Sq, d) / math.sqrt(d)
    scores = (q @ states(s["caches"][0], s["scales"][0]).transpose(2, 3)).reshape(B, Hkv, G, Sq, -1)
    step = torch.arange(Sq, device="cuda")
    last = (s["lens"] - s["new"])[:, None] + step  # the last key that each new token sees
    key = torch.arange(scores.shape[-1], device="cuda")
    seen = (key <= last[..., None]) & (key < s["lens"][:, None, None])
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = (scores - top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.reshape(B, Hkv, G * Sq, -1) @ states(s["caches"][1], s["scales"][1])).reshape(B, Hkv, G, Sq, d) / total
    lse = (top + total.log()).reshape(B, -1, Sq)
    live = (step < s["new"][:, None])[:, None]
    s["out"].copy_(torch.where(live[..., None], out.reshape(s["out"].shape).to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(live, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    s = state
    c = s["c"]
    if own:
        from long_context_sharded_gb300 import mercury as m
        if c["op"] == "rope":
            return m.mercury_rope(s["x"], s["plan"], s["pos"], inverse=c["inverse"], out=s["out"])
        if c["op"] == "append":
            m.mercury_kv_append(s["cache"], s["k"], s["v"], s["past"], new_lens=s["new"], rope=s["plan"], q=s["q"],
                                q_out=s["q_out"])
            return {"q": s["q_out"], "k_cache": s["caches"][0], "v_cache": s["caches"][1]}
        call = m.mercury_attn_paged_bf16 if c["bf16_out"] else m.mercury_attn_paged
        call(s["q"], s["cache"], s["lens"], new_lens=s["new"], causal=True, out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "rope":
        return s["out"].copy_(_rotated(s["x"], s["pos"], s["freq"], c, c["inverse"]).to(s["x"].dtype))
    return _plain_append(s) if c["op"] == "append" else _plain_attn(s)


# ------------------------------------------------------------------------------------- the definitions in 64 bits

def _turned64(x, pos, c, scaling, inverse=False):
    """The rotation as a product of complex numbers."""
    rot = c["rot"]
    rates, size = [], 1.0
    for i in range(rot // 2):
        base = ROPE_BASE * 4.0 ** (rot / (rot - 2.0)) if scaling == "ntk" else ROPE_BASE
        f = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == "linear":
            f /= 4.0
        if scaling == "yarn":
            turns = ROPE_ORIGINAL * f / (2.0 * math.pi)
            g = 0.0 if turns < 1.0 else 1.0 if turns > 32.0 else (turns - 1.0) / 31.0
            f, size = (1.0 - g) * f / 4.0 + g * f, 0.1 * math.log(4.0) + 1.0
        rates.append(-f if inverse else f)
    y = x.double().clone()
    at = torch.tensor([2 * i if c["interleaved"] else i for i in range(rot // 2)], device=x.device)
    to = at + (1 if c["interleaved"] else rot // 2)
    angle = pos.double().unsqueeze(1).unsqueeze(-1) * torch.tensor(rates, dtype=torch.float64, device=x.device)
    z = torch.complex(y[..., at], y[..., to]) * torch.polar(torch.full_like(angle, size), angle)
    y[..., at], y[..., to] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    if c["op"] == "rope" and c["B"] * c["H"] * c["S"] * c["d"] > 1 << 29:
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _turned64(s["x"], s["pos"], c, c["scaling"], c["inverse"])
    if c["op"] == "append":
        k_cache, v_cache, q_out = s["caches"][0].double(), s["caches"][1].double(), s["q_out"].double()
        past, new, table = s["past"].tolist(), s["new"].tolist(), s["table"]
        for b in range(c["B"]):
            n = new[b]
            at = torch.arange(past[b], past[b] + n, device="cuda")
            page, row = table[b].long()[torch.div(at, c["page"], rounding_mode="floor")], at % c["page"]
            k = _turned64(s["k"][b:b + 1, :, :n], at[None], c, "none")[0].transpose(0, 1)
            v = s["v"][b, :, :n].double().transpose(0, 1)
            if c["e4m3"]:
                k = (k / s["scales"][0].double()[:, None]).clamp(-448, 448)
                v = (v / s["scales"][1].double()[:, None]).clamp(-448, 448)
            k_cache[page, :, row], v_cache[page, :, row] = k, v
            q_out[b, :, :n] = _turned64(s["q"][b:b + 1, :, :n], at[None], c, "none")[0]
        return {"q": q_out, "k_cache": k_cache, "v_cache": v_cache}
    out, lse = s["out"].double(), s["lse"].double()
    lens, new, G = s["lens"].tolist(), s["new"].tolist(), c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        at = torch.arange(lens[b], device="cuda")
        page, row = s["table"][b].long()[torch.div(at, c["page"], rounding_mode="floor")], at % c["page"]
        for h in range(c["Hkv"]):
            k, v = (x.view(torch.uint8)[page, h, row].view(x.dtype) if c["e4m3"] else x[page, h, row] for x in s["caches"])
            k, v = k.double(), v.double()
            if c["e4m3"]:
                k, v = k * s["scales"][0][h].double(), v * s["scales"][1][h].double()
            for i in range(new[b]):
                n = lens[b] - new[b] + i + 1
                x = s["q"][b, h * G:(h + 1) * G, i].double() @ k[:n].T / math.sqrt(c["d"])
                lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, 1)
                out[b, h * G:(h + 1) * G, i] = torch.softmax(x, 1) @ v[:n]
    return {"out": out, "lse": lse}
