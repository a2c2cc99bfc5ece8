"""Measured cases of the operators around the NVFP4 linear layer: layer norm and
its gradient, the linear product with its fused epilogue, and the gradient of
that epilogue (activation and bias).

Each case runs in two forms.  With ``own`` false, ``run`` computes the operator
from elementary torch operations in 32 bits, rounded once at the end; with
``own`` true it makes the library's calls.  ``exact`` is the definition in 64
bits, written apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")  # in the order of the library's ACT_* codes
EPS = 1e-5


def listed():
    return [
        # one new token's hidden state, normalised before the quantizer: pure latency
        {"name": "norm_token", "op": "norm", "M": 1, "N": 5120, "x": "bf16", "y": "bf16", "amax": True},
        # a short prompt through an odd hidden size, from an fp32 residual stream
        {"name": "norm_ragged", "op": "norm", "M": 1237, "N": 2731, "x": "f32", "y": "bf16", "amax": False},
        # a training batch at the layer's hidden size, with the amax that the quantizer takes next
        {"name": "norm_train", "op": "norm", "M": 16384, "N": 5120, "x": "bf16", "y": "bf16", "amax": True},
        # fine-tuning of a small model on a short batch, everything in fp32
        {"name": "norm_grad_small", "op": "norm_grad", "M": 515, "N": 1023, "x": "f32", "y": "f32", "residual": False},
        # a training batch: the norm's gradient joined with the residual stream's
        {"name": "norm_grad_train", "op": "norm_grad", "M": 16384, "N": 5120, "x": "bf16", "y": "bf16",
         "residual": True},
        # one new token through the layer's first product: the weight's bytes are everything
        {"name": "linear_token", "op": "linear", "M": 1, "N": 20480, "K": 5120, "act": "gelu_tanh",
         "residual": False, "z": False, "amax": True, "out": "bf16"},
        # a batch of new tokens through the second product, added to the residual stream
        {"name": "linear_batch", "op": "linear", "M": 24, "N": 5120, "K": 20480, "act": "none",
         "residual": True, "z": False, "amax": False, "out": "bf16"},
        # a ragged prompt through a layer whose sizes fill no tile, kept in fp32
        {"name": "linear_ragged", "op": "linear", "M": 333, "N": 1000, "K": 1056, "act": "silu",
         "residual": False, "z": True, "amax": False, "out": "f32"},
        # training, first product: GELU, its input kept for the backward pass, amax for the next quantize
        {"name": "linear_train_up", "op": "linear", "M": 16384, "N": 20480, "K": 5120, "act": "gelu_tanh",
         "residual": False, "z": True, "amax": True, "out": "bf16"},
        # training, second product: bias and residual
        {"name": "linear_train_down", "op": "linear", "M": 16384, "N": 5120, "K": 20480, "act": "none",
         "residual": True, "z": False, "amax": False, "out": "bf16"},
        # gradient of bias and activation on a handful of tokens, odd width, fp32
        {"name": "act_grad_small", "op": "act_grad", "M": 67, "N": 1001, "t": "f32", "act": "silu"},
        # the same for a training batch at the layer's inner size
        {"name": "act_grad_train", "op": "act_grad", "M": 16384, "N": 20480, "t": "bf16", "act": "gelu_tanh"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "linear", "linear", "act_grad"))
    if op in ("norm", "norm_grad"):
        N = _log(rng, 48, 20480)
        M = _log(rng, 1, min(16384, 16384 * 5120 // N))
        x = rng.choice(("bf16", "f32"))
        y = "bf16" if x == "bf16" else rng.choice(("bf16", "f32"))
        c = {"op": op, "M": M, "N": N, "x": x, "y": y}
        if op == "norm":
            c["amax"] = rng.random() < 0.5 and y == "bf16"
        else:
            c["residual"] = rng.random() < 0.5
        return c
    if op == "linear":
        K = 32 * _log(rng, 2, 640)
        N = _log(rng, 40, 20480)
        M = _log(rng, 1, max(1, min(16384, 16384 * 20480 * 5120 // (N * K))))
        out = rng.choice(("bf16", "bf16", "f32"))
        return {"op": op, "M": M, "N": N, "K": K, "act": rng.choice(ACTS), "residual": rng.random() < 0.4,
                "z": rng.random() < 0.3, "amax": rng.random() < 0.3 and out == "bf16", "out": out}
    N = _log(rng, 48, 20480)
    return {"op": op, "M": _log(rng, 1, 16384), "N": N, "t": rng.choice(("bf16", "f32")) if N < 10240 else "bf16",
            "act": rng.choice(ACTS[1:])}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _hidden(M, N, g):
    """A residual stream: N(0, 1) around a small offset, a few channels thirty times as large."""
    x = torch.randn(M, N, generator=g, device=DEV)
    cols = torch.randint(0, N, (max(1, N // 2000),), generator=g, device=DEV)
    x[:, cols] *= 30.0
    return x + 0.1


def _gradient(M, N, g):
    """Student-t with three degrees of freedom, scaled by 1e-3: heavy tails, as gradients have them."""
    chi = torch.zeros(M, N, device=DEV)
    for _ in range(3):
        chi += torch.randn(M, N, generator=g, device=DEV).square_()
    return torch.randn(M, N, generator=g, device=DEV) / (chi / 3).sqrt_() * 1e-3


def _nvfp4(x):
    """x as an NVFP4 operand: packed codes, scale bytes in the tiled 128 x 4 layout, tensor scale."""
    R, K = x.shape
    alpha = x.abs().amax() / 2688.0
    blocks = x.view(R, K // 16, 16)
    s = (blocks.abs().amax(2) / (6.0 * alpha)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * alpha
    v = torch.where(d[:, :, None] > 0, blocks / d[:, :, None], torch.zeros((), device=x.device))
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(v.abs().contiguous(), steps, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(R, K // 2, 2)
    Rp, Cp = -(-R // 128) * 128, -(-(K // 16) // 4) * 4
    sf = torch.zeros(Rp, Cp, dtype=torch.uint8, device=x.device)
    sf[:R, :K // 16] = s.view(torch.uint8)
    sf = sf.view(Rp // 128, 4, 32, Cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(Rp, Cp)
    return code[:, :, 0] | (code[:, :, 1] << 4), sf, alpha.reshape(1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, M, N = case, case["M"], case["N"]
    s = dict(case)
    if c["op"] in ("norm", "norm_grad"):
        xt, yt = DTYPES[c["x"]], DTYPES[c["y"]]
        s["x"] = _hidden(M, N, g).to(xt)
        s["gamma"] = 1.0 + 0.1 * torch.randn(N, generator=g, device=DEV)
        s["beta"] = 0.02 * torch.randn(N, generator=g, device=DEV)
        if c["op"] == "norm_grad":
            s["dy"] = _gradient(M, N, g).to(yt)
            s["dres"] = _gradient(M, N, g).to(xt) if c["residual"] else None
            var, mean = torch.var_mean(s["x"].float(), dim=1, correction=0)  # what the forward pass saved
            s["mean"], s["rstd"] = mean, torch.rsqrt(var + EPS)
    elif c["op"] == "linear":
        K = c["K"]
        s["a"] = _nvfp4(_hidden(M, K, g).to(torch.bfloat16).float())
        s["b"] = _nvfp4((0.02 * torch.randn(N, K, generator=g, device=DEV)).to(torch.bfloat16).float())
        s["bias"] = 0.1 * torch.randn(N, generator=g, device=DEV)
        s["res"] = torch.randn(M, N, generator=g, device=DEV).to(DTYPES[c["out"]]) if c["residual"] else None
    else:
        t = DTYPES[c["t"]]
        s["dy"] = _gradient(M, N, g).to(t)
        s["z"] = (1.5 * torch.randn(M, N, generator=g, device=DEV)).to(t)
    return s


# ---- the plain form -------------------------------------------------------------------------------------------


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    y = (d * rstd * s["gamma"] + s["beta"]).to(DTYPES[s["y"]])
    out = {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["amax"]:
        out["amax"] = y.abs().amax().expand(2)
    return out


def _plain_norm_grad(s):
    dy, mean, rstd = s["dy"].float(), s["mean"][:, None], s["rstd"][:, None]
    xhat = (s["x"].float() - mean) * rstd
    gy = dy * s["gamma"]
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _plain_operand(q, sf, K):
    """Codes times block scales in fp32 (without the tensor scale)."""
    R = q.shape[0]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    grid = torch.cat([grid, -grid])
    v = grid[torch.stack([q & 15, q >> 4], 2).long()].view(R, K // 16, 16)
    Rp, Cp = sf.shape
    e = sf.view(Rp // 128, Cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(Rp, Cp)[:R, :K // 16]
    return (v * e.contiguous().view(torch.float8_e4m3fn).float()[:, :, None]).view(R, K)


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_linear(s):
    (qa, sa, aa), (qb, sb, ab) = s["a"], s["b"]
    z = (_plain_operand(qa, sa, s["K"]) @ _plain_operand(qb, sb, s["K"]).t()) * (aa * ab) + s["bias"]
    d = _plain_act(z, s["act"])
    if s["res"] is not None:
        d = d + s["res"].float()
    out = {"d": d.to(DTYPES[s["out"]])}
    if s["z"]:
        out["z"] = z.to(DTYPES[s["out"]])
    if s["amax"]:
        out["amax"] = out["d"].abs().amax().expand(2)
    return out


def _plain_act_grad(s):
    dy, z, act = s["dy"].float(), s["z"].float(), s["act"]
    if act == "relu":
        d = (z > 0).float()
    elif act == "gelu":
        d = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    elif act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        d = 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
        d = p * (1.0 + z * (1.0 - p))
    dz = dy * d
    return {"dz": dz.to(s["z"].dtype), "dbias": dz.sum(0)}


# ---- one pass -------------------------------------------------------------------------------------------------


def _amax16(a):
    """The fp32 amax pair at the type of the tensor it was taken from: its upper half, the lower being zero."""
    return a.view(torch.bfloat16)[1::2]


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "linear": _plain_linear,
                "act_grad": _plain_act_grad}[s["op"]](s)
    import nvfp4_bit_block_gb300 as nv
    if s["op"] == "norm":
        r = nv.nvfp4_layernorm(s["x"], s["gamma"], s["beta"], EPS, out_dtype=DTYPES[s["y"]], want_amax=s["amax"])
        out = {"y": r.y, "mean": r.mean, "rstd": r.rstd}
        if s["amax"]:
            out["amax"] = _amax16(r.amax)
        return out
    if s["op"] == "norm_grad":
        r = nv.nvfp4_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], dres=s["dres"])
        return {"dx": r.dx, "dgamma": r.dgamma, "dbeta": r.dbeta}
    if s["op"] == "linear":
        r = nv.nvfp4_linear(*s["a"], *s["b"], bias=s["bias"], act=ACTS.index(s["act"]), residual=s["res"],
                            out_dtype=DTYPES[s["out"]], want_z=s["z"], want_amax=s["amax"])
        out = {"d": r.d}
        if s["z"]:
            out["z"] = r.z
        if s["amax"]:
            out["amax"] = _amax16(r.amax)
        return out
    r = nv.nvfp4_act_backward(s["dy"], s["z"], ACTS.index(s["act"]))
    return {"dz": r.dz, "dbias": r.dbias}


def work(case):
    c, M, N = case, case["M"], case["N"]
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "norm":
        return {"bytes": M * N * (size[c["x"]] + size[c["y"]]) + 8 * N + 8 * M, "flops": 9 * M * N}
    if c["op"] == "norm_grad":
        per = size[c["y"]] + size[c["x"]] * (3 if c["residual"] else 2)
        return {"bytes": M * N * per + 8 * M + 12 * N, "flops": 15 * M * N}
    if c["op"] == "linear":
        K = c["K"]
        outs = 1 + (1 if c["residual"] else 0) + (1 if c["z"] else 0)
        return {"bytes": (M + N) * K * 9 / 16 + 4 * N + size[c["out"]] * M * N * outs, "flops": 2 * M * N * K}
    return {"bytes": M * N * 3 * size[c["t"]] + 4 * N, "flops": 20 * M * N}


# ---- the definition in 64 bits --------------------------------------------------------------------------------


def _value64(q, sf, K):
    """An operand's codes times its block scales, each decoded from its bits."""
    R = q.shape[0]
    b = q.to(torch.int32)
    v = torch.empty(R, K, dtype=torch.float64, device=q.device)
    for half in (0, 1):
        n = (b >> (4 * half)) & 15
        e, m = (n >> 1) & 3, n & 1
        mag = torch.where(e == 0, 0.5 * m.double(), torch.ldexp(1.0 + 0.5 * m.double(), (e - 1).double()))
        v[:, half::2] = torch.where(n >= 8, -mag, mag)
    r = torch.arange(R, device=q.device)[:, None]
    k = torch.arange(K // 16, device=q.device)[None, :]
    at = ((r // 128) * (sf.shape[1] // 4) + k // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4
    byte = sf.reshape(-1)[at].to(torch.int32)
    e, m = (byte >> 3) & 15, (byte & 7).double()
    scale = torch.where(e == 0, torch.ldexp(m, torch.full_like(m, -9)), torch.ldexp(1 + m / 8, (e - 7).double()))
    return (v.view(R, K // 16, 16) * scale[:, :, None]).view(R, K)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("norm", "norm_grad"):
        x = s["x"].double()
        mu = x.sum(1) / x.shape[1]
        c = x - mu[:, None]
        r = 1.0 / torch.sqrt((c * c).sum(1) / x.shape[1] + EPS)
        g = s["gamma"].double()
        if op == "norm":
            c *= r[:, None]
            y = torch.addcmul(s["beta"].double(), c, g)
            out = {"y": y, "mean": mu, "rstd": r}
            if s["amax"]:
                out["amax"] = torch.stack([y.abs().max()] * 2)
            return out
        # through the Jacobian of (x - mean) / std: subtract the parts along 1 and along xhat
        h = c * r[:, None]
        dy = s["dy"].double()
        w = dy * g
        along = (w * h).sum(1) / x.shape[1]
        dx = (w - (w.sum(1) / x.shape[1])[:, None] - along[:, None] * h) * r[:, None]
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("mn,mn->n", dy, h), "dbeta": dy.sum(0)}
    if op == "linear":
        K = s["K"]
        a, b = _value64(s["a"][0], s["a"][1], K), _value64(s["b"][0], s["b"][1], K)
        z = torch.einsum("mk,nk->mn", a, b)
        z.mul_(s["a"][2].double() * s["b"][2].double()).add_(s["bias"].double())
        d = {"none": lambda: z.clone(), "relu": lambda: z.clamp(min=0.0),
             "gelu": lambda: 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0)),
             "gelu_tanh": lambda: z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)),
             "silu": lambda: z * torch.sigmoid(z)}[s["act"]]()
        if s["res"] is not None:
            d += s["res"].double()
        out = {"d": d}
        if s["z"]:
            out["z"] = z
        if s["amax"]:
            out["amax"] = torch.stack([d.abs().max()] * 2)
        return out
    dy, z, act = s["dy"].double(), s["z"].double(), s["act"]
    if act == "relu":
        dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    elif act == "gelu":
        dz = dy * (0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    else:
        # act(z) = z * sigmoid(u(z)); derivative sigmoid + z * sigmoid * (1 - sigmoid) * u'
        k = 2.0 * math.sqrt(2.0 / math.pi)
        p = torch.sigmoid(z if act == "silu" else k * (z + 0.044715 * z ** 3))
        du = 1.0 if act == "silu" else k * (1.0 + 3 * 0.044715 * z ** 2)
        dz = dy * (p + z * p * (1.0 - p) * du)
    return {"dz": dz, "dbias": dz.sum(0)}
