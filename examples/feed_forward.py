"""A pre-norm feed-forward block on NVFP4, forward, backward and for one token:

    out = x + W2 gelu(W1 norm(x) + b1) + b2

Every matrix product runs on NVFP4 operands.  The norm and the first product hand
their output's amax to the quantizer, so that no tensor is read again for it; the
bias, the activation and the residual stream are in the products' epilogues; the
gradients of bias and activation and of the norm close the training step.

    python examples/feed_forward.py [--tokens 4096] [--hidden 5120] [--inner 20480]

prints the time of each pass and how far its results are from the same block in
fp32 without quantization.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import nvfp4_bit_block_gb300 as nv  # noqa: E402

BOTH = nv.ROWWISE | nv.COLWISE | nv.SF_SWIZZLED


def quantize(x, amax=None, flags=BOTH):
    """x as NVFP4 operands; `amax` where the kernel that made x has it."""
    return nv.nvfp4_quantize(x, nv.nvfp4_amax(x, flags) if amax is None else amax, flags)


def rows(q):
    """The operand with x's rows (K along its columns)."""
    return q.q_row, q.s_row, q.alpha[0:1]


def cols(q):
    """The operand with x's columns (K along its rows)."""
    return q.q_col, q.s_col, q.alpha[1:2]


class FeedForward:
    """Weights in bf16 (hidden and inner multiples of 32), their NVFP4 copies made once per step."""

    def __init__(self, hidden, inner, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)
        self.gamma = 1 + normal(hidden, std=0.1, dtype=torch.float32)
        self.beta = normal(hidden, std=0.02, dtype=torch.float32)
        self.w1, self.b1 = normal(inner, hidden, std=0.02), normal(inner, std=0.1, dtype=torch.float32)
        self.w2, self.b2 = normal(hidden, inner, std=0.02), normal(hidden, std=0.1, dtype=torch.float32)
        self.requantize()

    def requantize(self):
        self.q1, self.q2 = quantize(self.w1, flags=BOTH | nv.TWO_D), quantize(self.w2, flags=BOTH | nv.TWO_D)

    def forward(self, x, keep=True):
        """out, and what the backward pass needs.  x: tokens x hidden, bf16; with
        keep=False any number of tokens, else a multiple of 32."""
        flags = BOTH if keep else nv.ROWWISE | nv.SF_SWIZZLED
        n = nv.nvfp4_layernorm(x, self.gamma, self.beta, want_stats=keep, want_amax=True)
        qn = quantize(n.y, n.amax, flags)
        up = nv.nvfp4_linear(*rows(qn), *rows(self.q1), bias=self.b1, act=nv.ACT_GELU_TANH, want_z=keep, want_amax=True)
        qh = quantize(up.d, up.amax, flags)
        out = nv.nvfp4_linear(*rows(qh), *rows(self.q2), bias=self.b2, residual=x).d
        return out, ((x, n.mean, n.rstd, qn, up.z, qh) if keep else None)

    def backward(self, dout, saved):
        """Gradients of x and of the weights (fp32), from that of out."""
        x, mean, rstd, qn, z, qh = saved
        grads = {"b2": nv.nvfp4_act_backward(dout, None, nv.ACT_NONE, want_dz=False).dbias}
        qd = quantize(dout)
        grads["w2"] = nv.nvfp4_linear(*cols(qd), *cols(qh), out_dtype=torch.float32).d
        dh = nv.nvfp4_linear(*rows(qd), *cols(self.q2)).d
        t = nv.nvfp4_act_backward(dh, z, nv.ACT_GELU_TANH, out=dh)
        grads["b1"] = t.dbias
        qz = quantize(t.dz)
        grads["w1"] = nv.nvfp4_linear(*cols(qz), *cols(qn), out_dtype=torch.float32).d
        dn = nv.nvfp4_linear(*rows(qz), *cols(self.q1)).d
        g = nv.nvfp4_layernorm_backward(dn, x, mean, rstd, self.gamma, dres=dout, out=dn)
        grads.update(x=g.dx, gamma=g.dgamma, beta=g.dbeta)
        return grads

    def reference(self, x, dout):
        """The same block by torch in fp32: (out, gradients)."""
        F = torch.nn.functional
        p = {k: getattr(self, k).float().requires_grad_(True) for k in ("gamma", "beta", "w1", "b1", "w2", "b2")}
        p["x"] = x.float().requires_grad_(True)
        n = F.layer_norm(p["x"], (x.shape[1],), p["gamma"], p["beta"])
        out = p["x"] + F.linear(F.gelu(F.linear(n, p["w1"], p["b1"]), approximate="tanh"), p["w2"], p["b2"])
        out.backward(dout.float())
        return out.detach(), {k: v.grad for k, v in p.items()}


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def run(tokens, hidden, inner, timing=False):
    """Forward, backward and one-token pass; returns the relative distances from the fp32 block."""
    block = FeedForward(hidden, inner)
    x = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    dout = (torch.randn(tokens, hidden, device="cuda") * 1e-3).to(torch.bfloat16)
    out, saved = block.forward(x)
    grads = block.backward(dout, saved)
    one, _ = block.forward(x[:1], keep=False)
    want_out, want = block.reference(x, dout)
    far = {"out": off(out - x, want_out - x.float()), "one token": off(one - x[:1], (want_out - x.float())[:1])}
    far.update({"d" + k: off(v, want[k]) for k, v in grads.items()})
    if timing:
        for name, f in (("forward", lambda: block.forward(x)), ("backward", lambda: block.backward(dout, saved)),
                        ("one token", lambda: block.forward(x[:1], keep=False))):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            for k in range(13):
                if k == 3:
                    a.record()
                f()
            b.record()
            torch.cuda.synchronize()
            print(f"{name:10s} {a.elapsed_time(b) / 10 * 1e3:9.1f} us")
    return far


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--inner", type=int, default=20480)
    a = ap.parse_args()
    nv.build()
    for name, v in run(a.tokens, a.hidden, a.inner, timing=True).items():
        print(f"{name:10s} off by {v:.3f} of its norm (two NVFP4 operands per product)")
