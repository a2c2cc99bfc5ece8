"""The attention operators' formulas in plain torch (64 bits, or 32 where the definition
says so), for the tests of include/nvfp4_attention.h."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def turn64(x, positions, inv_freq, interleaved, back=False):
    """Pairs of the last axis turned; x: (T, H, D) in 64 bits."""
    R = inv_freq.numel()
    a = positions.double()[:, None] * inv_freq.double()[None, :]
    c, s = a.cos()[:, None, :], a.sin()[:, None, :] * (-1.0 if back else 1.0)
    i = torch.arange(R, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R)
    y = x.clone()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def pair_size64(x, inv_freq, interleaved):
    """|a| + |b| of each value's pair (|x| of what passes)."""
    R = inv_freq.numel()
    i = torch.arange(R, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R)
    m = x.abs()
    y = m.clone()
    y[..., ia] = y[..., ib] = m[..., ia] + m[..., ib]
    return y


def norm64(x, gamma, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if gamma is None else y * gamma.double()


def rope64(x, positions, inv_freq, gamma, eps, norm, interleaved):
    """(the result, the size of what entered each value)."""
    y = norm64(x, gamma, eps) if norm else x.double()
    return turn64(y, positions, inv_freq, interleaved), pair_size64(y, inv_freq, interleaved)


def rope_grad64(dy, x, positions, inv_freq, gamma, eps, norm, interleaved):
    """(dx, size of what entered it, dgamma, sum of its magnitudes)."""
    dy = dy.double()
    g = turn64(dy, positions, inv_freq, interleaved, back=True)
    gm = pair_size64(dy, inv_freq, interleaved)
    if not norm:
        return g, gm, None, None
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h = x * r
    w, wm = (g, gm) if gamma is None else (g * gamma.double(), gm * gamma.double().abs())
    dx = r * (w - h * (w * h).mean(-1, keepdim=True))
    size = r * (wm + h.abs() * (wm * h.abs()).mean(-1, keepdim=True))
    return dx, size, (g * h).sum((0, 1)), (gm * h.abs()).sum((0, 1))


def e4m3(t):
    """The scale byte of t >= 0 (fp32): nearest even, saturating at 448."""
    return t.clamp(max=448.0).to(torch.float8_e4m3fn)


def quantize32(x, alpha):
    """x (..., D) fp32 on the CPU as (codes 0..15 (..., D), scale values (..., D/16)): the
    definition's fp32 quotients."""
    x = x.float().cpu()
    limit = torch.finfo(torch.float32).max
    x = torch.where(x.isnan(), torch.zeros(()), x.clamp(-limit, limit))
    b = x.unflatten(-1, (-1, 16))
    alpha = torch.tensor(alpha, dtype=torch.float32)
    s = e4m3((b.abs().amax(-1) / (6.0 * alpha)).clamp(max=1e6)).float()
    d = (s * alpha)[..., None]
    v = torch.where(d > 0, b / torch.where(d > 0, d, torch.ones(())), torch.zeros(()))
    a = v.abs().double().unsqueeze(-1)
    dist = (a - GRID).abs()
    near = dist.min(-1, keepdim=True).values
    even = torch.tensor([0, 1, 0, 1, 0, 1, 0, 1]).double() * 0.25  # among the two nearest the even code
    code = torch.where(dist == near, even, torch.full_like(dist, 9.0)).argmin(-1)
    code = torch.where(a[..., 0] > 6.0, torch.full_like(code, 7), code)
    code = code | ((v < 0).long() << 3)
    return code.flatten(-2), s


def values64(codes, scales):
    """Packed codes (..., D/2) and scale bytes (..., D/16) without the tensor scale."""
    grid = torch.cat([GRID, -GRID]).to(codes.device)
    v = grid[torch.stack([codes & 15, codes >> 4], -1).long()].flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(16, -1)


def sequence64(cache, table, b, n):
    """Keys and values of the first n positions of sequence b: (n, heads, D) each; NaN where the
    page is out of range."""
    S = cache.k_codes.shape[2]
    out = []
    for i, (c, s) in enumerate(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))):
        at = torch.arange(n, device=c.device)
        page = table[b, at // S].long() if n else at
        ok = (page >= 0) & (page < c.shape[0])
        page = torch.where(ok, page, torch.zeros_like(page))
        x = values64(c[page, :, at % S], s[page, :, at % S]) * cache.alpha[i].double()
        x[~ok] = math.nan
        out.append(x)
    return out


def visible(n, m, causal, window, sinks, device):
    p = torch.arange(n - m, n, device=device)[:, None]
    j = torch.arange(n, device=device)[None, :]
    if not causal:
        return torch.ones((m, n), dtype=torch.bool, device=device)
    see = j <= p
    if window:
        see = see & ((p - j < window) | (j < sinks))
    return see


def attend64(q, cache, starts, lengths, table, scale=None, causal=True, window=0, sinks=0):
    """(o, lse, size of what entered o, size of what entered a score); rows of no sequence are NaN."""
    T, Hq, D = q.shape
    Hk = cache.k_codes.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    size, lse = o.clone(), o[..., 0].clone()
    score = lse.clone()
    starts, lengths = starts.tolist(), lengths.tolist()
    for b, n in enumerate(lengths):
        m = starts[b + 1] - starts[b]
        if m == 0:
            continue
        rows = slice(starts[b], starts[b + 1])
        k, v = sequence64(cache, table, b, n)
        ok = ~k[:, 0, 0].isnan()
        k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
        see = visible(n, m, causal, window, sinks, q.device) & ok[None, :]
        for h in range(Hq):
            qh, kh, vh = q[rows, h].double(), k[:, h // G], v[:, h // G]
            s = (qh @ kh.t()) * scale
            s = s.masked_fill(~see, -math.inf)
            top = s.amax(-1, keepdim=True) if n else torch.full((m, 1), -math.inf, device=q.device)
            top = torch.where(top.isinf() & (top < 0), torch.zeros_like(top), top)
            e = torch.exp(s - top)
            total = e.sum(-1, keepdim=True)
            w = torch.where(total > 0, e / total.clamp(min=1e-300), torch.zeros_like(e))
            o[rows, h] = w @ vh
            size[rows, h] = w @ vh.abs() + 2.0 ** -14 * torch.where(see, 1.0, 0.0).double() @ vh.abs()
            lse[rows, h] = torch.where(total > 0, top + total.log(), torch.full_like(total, -math.inf))[:, 0]
            mag = ((qh.abs() @ kh.abs().t()) * abs(scale)).masked_fill(~see, 0.0)
            score[rows, h] = mag.amax(-1) if n else 0.0
    return o, lse, size, score
