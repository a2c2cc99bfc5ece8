"""A pre-norm attention block on NVFP4, taking prompts in and answering token by token:

    out = x + Wo attention(rotate(norm(Wq n)), rotate(norm(Wk n)), Wv n),  n = norm(x)

The matrix products run on NVFP4 operands and the keys and values stay in a paged cache
of 4-bit codes.  Queries and keys are normalised and rotated where the product left them.

    python examples/attention_block.py [--hidden 5120] [--heads 40] [--kv-heads 8] [--prompt 2048]

prints the time of a prompt and of a next token, and how far the results are from the same
block in fp32 without quantization.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import nvfp4_bit_block_gb300 as nv  # noqa: E402

FLAGS = nv.ROWWISE | nv.SF_SWIZZLED


def operand(x, amax=None, flags=FLAGS):
    """x's rows as an NVFP4 operand; `amax` where the kernel that made x has it."""
    q = nv.nvfp4_quantize(x, nv.nvfp4_amax(x, flags) if amax is None else amax, flags)
    return q.q_row, q.s_row, q.alpha[0:1]


class AttentionBlock:
    def __init__(self, hidden, heads, kv_heads, dim=128, base=10000.0, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.gamma = 1 + normal(hidden, std=0.1, dtype=torch.float32)
        self.beta = normal(hidden, std=0.02, dtype=torch.float32)
        self.gamma_q, self.gamma_k = (1 + normal(dim, std=0.1, dtype=torch.float32) for _ in range(2))
        self.wqkv = normal((heads + 2 * kv_heads) * dim, hidden, std=0.02)
        self.wo = normal(hidden, heads * dim, std=0.02)
        self.inv_freq = (base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)).float()
        self.qqkv, self.qo = operand(self.wqkv, flags=FLAGS | nv.TWO_D), operand(self.wo, flags=FLAGS | nv.TWO_D)

    def forward(self, x, positions, cache, batch, window=0, sinks=0):
        """x: new tokens (rows as in `batch`) x hidden, bf16; their keys and values go into the cache."""
        T = x.shape[0]
        n = nv.nvfp4_layernorm(x, self.gamma, self.beta, want_stats=False, want_amax=True)
        qkv = nv.nvfp4_linear(*operand(n.y, n.amax), *self.qqkv).d.view(T, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        nv.nvfp4_qk_rope(q, k, positions, self.inv_freq, self.gamma_q, self.gamma_k, out_q=q, out_k=k)
        nv.nvfp4_cache_write(k, v, cache, *batch)
        a = nv.nvfp4_cache_attention(q, cache, *batch, window=window, sinks=sinks)
        return nv.nvfp4_linear(*operand(a.o.view(T, -1)), *self.qo, residual=x).d

    def reference(self, x, lengths, window=0, sinks=0):
        """The same block by torch in fp32 over whole sequences (rows one after another)."""
        F = torch.nn.functional
        n = F.layer_norm(x.float(), (x.shape[1],), self.gamma, self.beta)
        qkv = F.linear(n, self.wqkv.float()).view(x.shape[0], -1, self.dim)
        out, at = [], 0
        for length in lengths:
            q, k, v = qkv[at:at + length].split((self.heads, self.kv_heads, self.kv_heads), 1)
            pos = torch.arange(length, device=x.device)
            angle = pos.double()[:, None] * self.inv_freq.double()
            cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

            def turned(t, gamma):
                t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * gamma
                a, b = t.chunk(2, -1)
                return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            q, k = turned(q, self.gamma_q), turned(k, self.gamma_k)
            k, v = (t.repeat_interleave(self.heads // self.kv_heads, 1) for t in (k, v))
            see = pos[None, :] <= pos[:, None]
            if window:
                see &= (pos[:, None] - pos[None, :] < window) | (pos[None, :] < sinks)
            s = torch.einsum("ihd,jhd->hij", q, k) * self.dim ** -0.5
            p = s.masked_fill(~see, -torch.inf).softmax(-1)
            out.append(torch.einsum("hij,jhd->ihd", p, v).flatten(1))
            at += length
        return x.float() + F.linear(torch.cat(out), self.wo.float())


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(hidden, heads, kv_heads, prompts, answers=3, dim=128, page_size=16, window=0, sinks=0, timing=False):
    """Prompts of these lengths, then `answers` more tokens for each, one at a time; the relative distance of the
    block's change to x from the fp32 block's, for the prompts and for the answers."""
    block = AttentionBlock(hidden, heads, kv_heads, dim)
    B, ends = len(prompts), [n + answers for n in prompts]
    xs = [torch.randn(n, hidden, device="cuda").to(torch.bfloat16) for n in ends]
    width = max(-(-n // page_size) for n in ends)
    pages = torch.randperm(B * width, device="cuda").to(torch.int32).view(B, width)
    cache = nv.nvfp4_kv_cache(B * width, kv_heads, page_size, dim, (2.0 ** -7, 2.0 ** -7))
    starts = [0]
    for n in prompts:
        starts.append(starts[-1] + n)
    positions = ints([j for n in prompts for j in range(n)])
    x = torch.cat([t[:n] for t, n in zip(xs, prompts)])
    batch = (ints(starts), ints(prompts), pages)
    out = block.forward(x, positions, cache, batch, window, sinks)
    steps = []
    for k in range(answers):
        one = torch.stack([t[n + k] for t, n in zip(xs, prompts)])
        lengths = ints([n + k + 1 for n in prompts])
        steps.append((one, block.forward(one, lengths - 1, cache, (ints(list(range(B + 1))), lengths, pages), window, sinks)))
    want = block.reference(torch.cat(xs), ends, window, sinks)
    first = [0]
    for n in ends:
        first.append(first[-1] + n)
    wp = torch.cat([want[first[b]:first[b] + n] for b, n in enumerate(prompts)])
    far = {"prompts": off(out - x, wp - x.float())}
    if answers:
        wa = torch.cat([torch.stack([want[first[b] + n + k] for b, n in enumerate(prompts)]) for k in range(answers)])
        xa = torch.cat([s[0] for s in steps])
        far["answers"] = off(torch.cat([s[1] for s in steps]) - xa, wa - xa.float())
    if timing:
        last = (steps[-1][0], ints(ends) - 1, cache, (ints(list(range(B + 1))), ints(ends), pages), window, sinks)
        for name, f in (("prompts", lambda: block.forward(x, positions, cache, batch, window, sinks)),
                        ("next token", lambda: block.forward(*last))):
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
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--heads", type=int, default=40)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=2048)
    a = ap.parse_args()
    nv.build()
    for name, v in run(a.hidden, a.heads, a.kv_heads, [a.prompt], timing=True).items():
        print(f"{name:10s} off by {v:.3f} of its norm (NVFP4 operands, keys and values)")
