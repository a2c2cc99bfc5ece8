"""Measured cases of the attention operators on an NVFP4 cache of keys and values:
the norm and rotation of queries and keys and its gradient, the write into the
paged 4-bit cache, reading it back, and the attention that reads it.

Each case runs in two forms.  With ``own`` false, ``run`` computes the operator
from elementary torch operations in 32 bits (angles in 64), rounded once at the
end; with ``own`` true it makes the library's calls.  ``exact`` is the definition
in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
GOLDEN = 0.6180339887498949


def listed():
    heads = {"Hq": 40, "Hkv": 8, "D": 128}  # the layer's hidden size of 5120 in heads of 128, five queries to a key
    return [
        # one new token's queries and keys, before they reach the cache: pure latency
        {"name": "rope_token", "op": "rope", "T": 1, **heads, "R": 128, "pairs": "half", "x": "bf16", "y": "bf16",
         "norm": True, "far": 700},
        # a training batch, forward
        {"name": "rope_train", "op": "rope", "T": 16384, **heads, "R": 128, "pairs": "half", "x": "bf16", "y": "bf16",
         "norm": True, "far": 4096},
        # fine-tuning of a small model on a short batch in fp32: odd heads, half of each head rotated, neighbours paired
        {"name": "rope_grad_small", "op": "rope_grad", "T": 515, "Hq": 9, "Hkv": 3, "D": 96, "R": 48,
         "pairs": "neighbours", "x": "f32", "y": "f32", "norm": True, "far": 1030},
        # a training batch, backward, with the gradients of both norms' weights
        {"name": "rope_grad_train", "op": "rope_grad", "T": 16384, **heads, "R": 128, "pairs": "half", "x": "bf16",
         "y": "bf16", "norm": True, "far": 4096},
        # a batch of new tokens, one to a sequence, written and looked at again
        {"name": "write_batch", "op": "write", "B": 24, "len": 4096, "new": 1, "Hkv": 8, "D": 128, "page": 16,
         "x": "bf16"},
        # the keys and values of four long prompts, of uneven lengths
        {"name": "write_prompts", "op": "write", "B": 4, "len": 8192, "new": 8192, "Hkv": 8, "D": 128, "page": 64,
         "x": "bf16"},
        # the last tokens of a few short sequences, taken out in fp32 to be compared
        {"name": "read_short", "op": "read", "B": 7, "len": 333, "new": 61, "Hkv": 3, "D": 96, "page": 48, "y": "f32"},
        # a shared context taken out of the cache whole, for a kernel that wants it in bf16
        {"name": "read_context", "op": "read", "B": 1, "len": 65536, "new": 65536, "Hkv": 8, "D": 128, "page": 64,
         "y": "bf16"},
        # the next token of one conversation: latency
        {"name": "attend_token", "op": "attend", "B": 1, "len": 700, "new": 1, **heads, "page": 16, "window": 0,
         "sinks": 0},
        # the next token of a batch of uneven conversations: the cache's bytes are everything
        {"name": "attend_batch", "op": "attend", "B": 48, "len": 16384, "new": 1, **heads, "page": 64, "window": 0,
         "sinks": 0},
        # four drafted tokens a sequence, through a layer that sees a window and the first tokens
        {"name": "attend_window", "op": "attend", "B": 16, "len": 9000, "new": 4, **heads, "page": 32, "window": 2048,
         "sinks": 4},
        # prompts being taken in behind what the cache already holds: matrix products bound it
        {"name": "attend_prompts", "op": "attend", "B": 3, "len": 8192, "new": 2731, **heads, "page": 64, "window": 0,
         "sinks": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("rope", "rope_grad", "write", "read", "attend", "attend", "attend"))
    D = rng.choice((64, 96, 128, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op in ("rope", "rope_grad"):
        x = rng.choice(("bf16", "f32"))
        y = "bf16" if x == "bf16" else rng.choice(("bf16", "f32"))
        return {"op": op, "T": _log(rng, 1, min(16384, 16384 * 48 * 128 // (Hkv * (G + 1) * D))), "Hq": G * Hkv,
                "Hkv": Hkv, "D": D, "R": rng.choice((D, D, D // 2, D - 20)), "pairs": rng.choice(("half", "neighbours")),
                "x": x, "y": y, "norm": rng.random() < 0.7, "far": _log(rng, 700, 1000000)}
    page = rng.choice((16, 32, 48, 64, 128))
    if op in ("write", "read"):
        room = 32768 * 1024 // (Hkv * D)  # tokens, no more values than the largest listed case
        B = _log(rng, 1, 32)
        length = _log(rng, 1, min(65536, max(1, room // B)))
        new = rng.choice((1, length, _log(rng, 1, length)))
        c = {"op": op, "B": B, "len": length, "new": new, "Hkv": Hkv, "D": D, "page": page}
        c["x" if op == "write" else "y"] = rng.choice(("bf16", "bf16", "f32"))
        return c
    B = _log(rng, 1, 48)
    length = _log(rng, 1, min(65536, 48 * 16384 * 1024 // (B * Hkv * D)))
    pairs = 2 * 2731 * 8192 * 40 * 128 // (B * length * G * Hkv * D)
    new = min(length, rng.choice((1, 1, _log(rng, 1, 8), _log(rng, 1, 4096))), max(1, pairs))
    window = rng.choice((0, 0, _log(rng, 64, 4096)))
    return {"op": op, "B": B, "len": length, "new": new, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "page": page,
            "window": window, "sinks": rng.choice((0, 4, 17)) if window else 0}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _lengths(case):
    """Each sequence's length in the cache and how many of its last tokens are new: uneven where there are several;
    with more than eight sequences one slot of the batch is idle."""
    lens, news = [], []
    for i in range(case["B"]):
        share = 1.0 if i == 0 else 0.125 + 0.875 * ((i * GOLDEN) % 1.0)
        n = max(1, int(case["len"] * share))
        m = case["new"] if case["new"] <= 8 else max(1, int(case["new"] * share))
        lens.append(n)
        news.append(min(n, m) if case["B"] <= 8 or i != 5 else 0)
    return lens, news


def _starts(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return s


def _heads(T, H, D, g, spread=1.0):
    """Projected tokens: normal values, a few channels of each head many times as large, as keys have them."""
    x = torch.randn(T, H, D, generator=g, device=DEV) * spread
    cols = torch.randint(0, D, (H, max(1, D // 64)), generator=g, device=DEV)
    gain = torch.ones(H, D, device=DEV).scatter_(1, cols, 6.0)
    return x.mul_(gain)


def _gradient(shape, g):
    """Student-t with three degrees of freedom, scaled by 1e-3: heavy tails, as gradients have them."""
    chi = torch.zeros(shape, device=DEV)
    for _ in range(3):
        chi += torch.randn(shape, generator=g, device=DEV).square_()
    return torch.randn(shape, generator=g, device=DEV) / (chi / 3).sqrt_() * 1e-3


ALPHA = (0.03125, 0.015625)  # tensor scales of keys and values, fixed before the values are known: powers of two


def _codes(x, alpha):
    """x (..., D) in 4 bits: packed E2M1 codes (..., D/2) and E4M3 scale bytes (..., D/16)."""
    blocks = x.unflatten(-1, (-1, 16))
    s = (blocks.abs().amax(-1) / (6.0 * alpha)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * alpha
    v = torch.where(d[..., None] > 0, blocks / d[..., None], torch.zeros((), device=x.device))
    a = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=x.device)
    for border, even in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False),
                         (5.0, True)):  # a tie goes to the even code
        code += (a > border) if even else (a >= border)
    code |= (v < 0).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _slots(state, only_new):
    """Page and row of the cache of every (new) token, sequence after sequence."""
    page = state["page"]
    rows = []
    for b, (n, m) in enumerate(zip(state["lens"], state["news"])):
        at = torch.arange(n - m if only_new else 0, n, device=DEV)
        rows.append(state["pages"][b, at // page].long() * page + at % page)
    return torch.cat(rows)


def _cache(case, s, g, filled):
    """Pages in a random order, as a cache that has been in use has them; beyond a sequence's end they hold old bytes."""
    Hkv, D, page, lens = case["Hkv"], case["D"], case["page"], s["lens"]
    used = [-(-n // page) for n in lens]
    total = sum(used) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(case["B"], max(used), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    s["pages"] = table
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["starts"] = torch.tensor(_starts(s["news"]), dtype=torch.int32, device=DEV)
    s["alpha"] = torch.tensor(ALPHA, device=DEV)
    for name in ("k", "v"):
        s[name + "_codes"] = torch.randint(0, 256, (total, Hkv, page, D // 2), generator=g, device=DEV, dtype=torch.uint8)
        s[name + "_scales"] = torch.randint(0, 126, (total, Hkv, page, D // 16), generator=g, device=DEV,
                                            dtype=torch.uint8)
    if not filled:
        return
    slots = _slots(s, only_new=False)
    for i, name in enumerate(("k", "v")):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        for first in range(0, slots.numel(), 65536):
            part = slots[first:first + 65536]
            q, e = _codes(_heads(part.numel(), Hkv, D, g).to(torch.bfloat16).float(), ALPHA[i])
            codes[part // page, :, part % page] = q
            scales[part // page, :, part % page] = e


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, s = case, dict(case)
    if c["op"] in ("rope", "rope_grad"):
        T, Hq, Hkv, D, R = (c[n] for n in ("T", "Hq", "Hkv", "D", "R"))
        packed = _heads(T, Hq + 2 * Hkv, D, g).to(DTYPES[c["x"]])  # one product gives queries, keys and values
        s["q"], s["k"] = packed[:, :Hq], packed[:, Hq:Hq + Hkv]
        s["positions"] = ((torch.arange(T, device=DEV) + torch.randint(0, c["far"], (1,), generator=g, device=DEV))
                          % c["far"]).to(torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)).float()
        if c["norm"]:
            s["gamma_q"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
            s["gamma_k"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
        else:
            s["gamma_q"] = s["gamma_k"] = None
        if c["op"] == "rope_grad":
            s["dq"] = _gradient((T, Hq, D), g).to(DTYPES[c["y"]])
            s["dk"] = _gradient((T, Hkv, D), g).to(DTYPES[c["y"]])
        return s
    s["lens"], s["news"] = _lengths(c)
    T = sum(s["news"])
    _cache(c, s, g, filled=c["op"] != "write")
    if c["op"] == "write":
        s["k"] = _heads(T, c["Hkv"], c["D"], g).to(DTYPES[c["x"]])
        s["v"] = _heads(T, c["Hkv"], c["D"], g).to(DTYPES[c["x"]])
    elif c["op"] == "attend":
        s["q"] = torch.randn(T, c["Hq"], c["D"], generator=g, device=DEV).to(torch.bfloat16)
    if own:
        import nvfp4_bit_block_gb300 as nv
        s["cache"] = nv.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["alpha"])
    return s


# ---- the plain form -------------------------------------------------------------------------------------------


def _plain_angles(s):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _plain_rotate(x, cos, sin, s):
    """Pairs of the first R values of each head turned by their angles."""
    R = s["R"]
    if s["pairs"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., R:]], -1)


def _plain_rope(s):
    cos, sin = _plain_angles(s)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if s["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["gamma_" + name]
        out[name] = _plain_rotate(x, cos, sin, s).to(DTYPES[s["y"]])
    return out


def _plain_rope_grad(s):
    cos, sin = _plain_angles(s)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        g = _plain_rotate(s["d" + name].float(), cos, -sin, s)  # turned back
        if s["norm"]:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            xhat = x * r
            out["dgamma_" + name] = (g * xhat).sum((0, 1))
            g = g * s["gamma_" + name]
            g = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        out["d" + name] = g.to(s[name].dtype)
    return out


def _plain_values(codes, scales):
    """Codes times block scales in fp32 (without the tensor scale)."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    v = grid[torch.stack([codes & 15, codes >> 4], -1).long()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_gather(s, slots, name):
    page, i = s["page"], 0 if name == "k" else 1
    codes, scales = s[name + "_codes"], s[name + "_scales"]
    return _plain_values(codes[slots // page, :, slots % page], scales[slots // page, :, slots % page]) * s["alpha"][i]


def _plain_write(s):
    slots, page = _slots(s, only_new=True), s["page"]
    out = {}
    for i, name in enumerate(("k", "v")):
        q, e = _codes(s[name].float(), s["alpha"][i])
        s[name + "_codes"][slots // page, :, slots % page] = q
        s[name + "_scales"][slots // page, :, slots % page] = e
        out[name] = _plain_gather(s, slots, name).to(DTYPES[s["x"]])
    return out


def _plain_read(s):
    slots = _slots(s, only_new=True)
    return {name: _plain_gather(s, slots, name).to(DTYPES[s["y"]]) for name in ("k", "v")}


def _visible(s, n, m):
    """(new tokens, keys): key j is seen from position p if j <= p and it is in the window or one of the first."""
    p = torch.arange(n - m, n, device=DEV)[:, None]
    j = torch.arange(n, device=DEV)[None, :]
    see = j <= p
    if s["window"]:
        see &= (p - j < s["window"]) | (j < s["sinks"])
    return see


def _plain_attend(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G = Hq // Hkv
    slots = _slots(s, only_new=False)
    outs, lses, at, first = [], [], 0, 0
    for n, m in zip(s["lens"], s["news"]):
        if m:
            k, v = (_plain_gather(s, slots[first:first + n], name).transpose(0, 1) for name in ("k", "v"))
            q = s["q"][at:at + m].float().view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D)
            t = (q @ k.transpose(1, 2)).view(Hkv, G, m, n) * D ** -0.5
            t = t.masked_fill_(~_visible(s, n, m), -math.inf)
            top = t.amax(-1, keepdim=True)
            t = t.sub_(top).exp_()
            total = t.sum(-1, keepdim=True)
            o = (t.view(Hkv, G * m, n) @ v).view(Hkv, G, m, D) / total
            outs.append(o.permute(2, 0, 1, 3).reshape(m, Hq, D))
            lses.append((top + total.log()).squeeze(-1).permute(2, 0, 1).reshape(m, Hq))
        at, first = at + m, first + n
    return {"o": torch.cat(outs).to(torch.bfloat16), "lse": torch.cat(lses)}


# ---- one pass -------------------------------------------------------------------------------------------------


def run(state):
    s = state
    if not own:
        return {"rope": _plain_rope, "rope_grad": _plain_rope_grad, "write": _plain_write, "read": _plain_read,
                "attend": _plain_attend}[s["op"]](s)
    import nvfp4_bit_block_gb300 as nv
    if s["op"] == "rope":
        r = nv.nvfp4_qk_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["gamma_q"], s["gamma_k"],
                             eps=EPS, norm=s["norm"], interleaved=s["pairs"] == "neighbours", out_dtype=DTYPES[s["y"]])
        return {"q": r.q, "k": r.k}
    if s["op"] == "rope_grad":
        r = nv.nvfp4_qk_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["inv_freq"], s["gamma_q"],
                                      s["gamma_k"], eps=EPS, norm=s["norm"], interleaved=s["pairs"] == "neighbours")
        out = {"dq": r.dq, "dk": r.dk}
        if s["norm"]:
            out.update(dgamma_q=r.dgamma_q, dgamma_k=r.dgamma_k)
        return out
    batch = (s["starts"], s["lengths"], s["pages"])
    if s["op"] == "write":
        nv.nvfp4_cache_write(s["k"], s["v"], s["cache"], *batch)
        r = nv.nvfp4_cache_read(s["cache"], *batch, tokens=s["k"].shape[0], out_dtype=DTYPES[s["x"]])
        return {"k": r.k, "v": r.v}
    if s["op"] == "read":
        r = nv.nvfp4_cache_read(s["cache"], *batch, tokens=sum(s["news"]), out_dtype=DTYPES[s["y"]])
        return {"k": r.k, "v": r.v}
    r = nv.nvfp4_cache_attention(s["q"], s["cache"], *batch, window=s["window"], sinks=s["sinks"], want_lse=True)
    return {"o": r.o, "lse": r.lse}


def work(case):
    c, size = case, {"bf16": 2, "f32": 4}
    if c["op"] in ("rope", "rope_grad"):
        T, R = c["T"], c["R"]
        n = T * (c["Hq"] + c["Hkv"]) * c["D"]
        small = 4 * T + 2 * R + (8 * c["D"] if c["norm"] else 0)
        if c["op"] == "rope":
            return {"bytes": n * (size[c["x"]] + size[c["y"]]) + small, "flops": 8 * n}
        reads = size[c["y"]] + size[c["x"]] * (2 if c["norm"] else 1)  # without a norm the gradient needs no input
        return {"bytes": n * reads + small + (8 * c["D"] if c["norm"] else 0), "flops": 16 * n}
    lens, news = _lengths(c)
    D, Hkv = c["D"], c["Hkv"]
    row = 2 * Hkv * (D // 2 + D // 16)  # a token's keys and values in the cache
    if c["op"] == "write":  # the values come in, go into the cache and are looked at
        return {"bytes": sum(news) * (4 * Hkv * D * size[c["x"]] + 2 * row), "flops": 12 * sum(news) * Hkv * D}
    if c["op"] == "read":
        return {"bytes": sum(news) * (2 * Hkv * D * size[c["y"]] + row), "flops": 4 * sum(news) * Hkv * D}
    keys = pairs = 0
    for n, m in zip(lens, news):
        if m == 0:
            continue
        W, S = c["window"] or n, c["sinks"] if c["window"] else 0
        low = max(0, n - m + 1 - W)  # the first key in the window of the first new token
        keys += n - low + min(S, low)
        for p in range(n - m, n):
            first = max(0, p + 1 - W)
            pairs += p + 1 - first + min(S, first)
    return {"bytes": keys * row + sum(news) * c["Hq"] * (4 * D + 4), "flops": 4 * pairs * c["Hq"] * D}


# ---- the definition in 64 bits --------------------------------------------------------------------------------


def _turn64(x, positions, inv_freq, pairs, back):
    """The rotation as a product of complex numbers."""
    R = 2 * inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       positions.double()[:, None, None] * inv_freq.double())
    if back:
        turn = turn.conj()
    y = x.clone()
    first, second = (slice(0, R // 2), slice(R // 2, R)) if pairs == "half" else (slice(0, R, 2), slice(1, R, 2))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _nearest64(x, alpha):
    """x (..., D) as the cache holds it: the nearest E4M3 number to max / (6 alpha) for each 16 values, then the
    nearest of the eight magnitudes, a tie to the one with an even code."""
    b = x.unflatten(-1, (-1, 16))
    t = b.abs().amax(-1) / (6.0 * alpha)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)  # spacing of E4M3 at t
    scale = torch.clamp(torch.round(t / step) * step, max=448.0)            # round: ties to even
    d = (scale * alpha)[..., None]
    r = torch.where(d > 0, b.abs() / torch.where(d > 0, d, 1.0), 0.0).clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(r.clamp(min=1.0))) - 1)        # spacing of E2M1 at r
    return (torch.sign(b) * torch.clamp(torch.round(r / step) * step, max=6.0) * d).flatten(-2)


def _value64(codes, scales, alpha):
    """Cached values from their bits."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.ldexp(1 + 0.5 * m, (e - 1).double()))
    v = torch.where(n >= 8, -v, v)
    b = scales.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    f = torch.where(e == 0, torch.ldexp(m, torch.full_like(m, -9)), torch.ldexp(1 + m / 8, (e - 7).double()))
    return v * f.repeat_interleave(16, -1) * alpha


def _token64(s, b, first, last, name):
    """Tokens first .. last - 1 of sequence b, page by page."""
    page, alpha = s["page"], ALPHA[0 if name == "k" else 1]
    parts = []
    for p in range(first // page, -(-last // page)):
        at = int(s["table"][b][p])
        lo, hi = max(first - p * page, 0), min(last - p * page, page)
        parts.append((s[name + "_codes"][at, :, lo:hi], s[name + "_scales"][at, :, lo:hi]))
    codes, scales = torch.cat([q for q, _ in parts], 1), torch.cat([e for _, e in parts], 1)
    return _value64(codes, scales, alpha)  # heads, tokens, values


def _attend64(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G, at = Hq // Hkv, 0
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, (n, m) in enumerate(zip(s["lens"], s["news"])):
        if m == 0:
            continue
        k, v = _token64(s, b, 0, n, "k"), _token64(s, b, 0, n, "v")
        pos = torch.arange(n - m, n, device=DEV)
        key = torch.arange(n, device=DEV)
        hidden = key[None, :] > pos[:, None]
        if s["window"]:
            hidden |= (key[None, :] <= pos[:, None] - s["window"]) & (key[None, :] >= s["sinks"])
        bias = torch.zeros(m, n, dtype=torch.float64, device=DEV).masked_fill_(hidden, -math.inf)
        for h in range(Hq):
            logits = torch.addmm(bias, s["q"][at:at + m, h].double(), k[h // G].t(), alpha=1.0 / math.sqrt(D))
            z = torch.logsumexp(logits, 1)
            lse[at:at + m, h] = z
            o[at:at + m, h] = torch.exp(logits.sub_(z[:, None])) @ v[h // G]
        at += m
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rope":
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            if s["norm"]:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / s["D"] + EPS) * s["gamma_" + name].double()
            out[name] = _turn64(x, s["positions"], s["inv_freq"], s["pairs"], False)
        return out
    if op == "rope_grad":
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            dy = _turn64(s["d" + name].double(), s["positions"], s["inv_freq"], s["pairs"], True)
            if not s["norm"]:
                out["d" + name] = dy
                continue
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / s["D"] + EPS)
            w = dy * s["gamma_" + name].double()
            # d(x / rms) = dx / rms - x (x . dx) / (D rms^3)
            out["d" + name] = w / rms - x * ((w * x).sum(-1, keepdim=True) / (s["D"] * rms ** 3))
            out["dgamma_" + name] = torch.einsum("thd,thd->d", dy, x / rms)
        return out
    if op == "write":
        return {name: _nearest64(s[name].double(), ALPHA[i]) for i, name in enumerate(("k", "v"))}
    s["table"] = s["pages"].tolist()
    if op == "read":
        return {name: torch.cat([_token64(s, b, n - m, n, name).transpose(0, 1)
                                 for b, (n, m) in enumerate(zip(s["lens"], s["news"])) if m])
                for name in ("k", "v")}
    return _attend64(s)
