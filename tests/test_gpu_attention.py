"""The attention operators on the GPU, against their formulas in 64 bits (attention_oracle.py).

Tolerances.  u = 2^-24 is the rounding of an fp32 operation, u_out that of the result.
Norm and rotation: a sum of up to 512 squares in chains of at most 21 roundings is off by
2^-19.6 of itself, its root by half of that; the root, the products and the sine and cosine
(an argument rounded to 2^-25 half turns, 2 units in the result) add less than 2^-20: T_ROPE =
2^-18 of |a| + |b|, the pair's sizes.  The sums over rows add chains of at most 2^7 at the sizes
used here to that: T_SUM = 2^-16 of the sum of magnitudes.
Cache: codes and scales are exact, values rounded as the definition says.
Attention: a score is held to 2^-16 of sum |q k| scale (the bar of the GEMM's tests), which
moves each weight and their sum by that much, d; the base-2 exponential and its argument add
2^-18, and weights are rounded to fp16 where they meet the values: 2^-11 of the weight, or
2^-25 of the largest for small ones (in `size`, as 2^-14 * 2^-11 of sum |v|).  So o is
held to u_out |o| + (2^-11 + 2^-14 + 2 d) size and lse to d + 2^-17 + 2 u |lse|.
"""
import math

import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from attention_oracle import attend64, quantize32, rope64, rope_grad64, sequence64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U_OUT = {t: torch.finfo(t).eps / 2 for t in (BF, F32)}
T_ROPE, T_SUM, T_SCORE, T_WEIGHT = 2.0 ** -18, 2.0 ** -16, 2.0 ** -16, 2.0 ** -11 + 2.0 ** -14
TYPES = [(BF, BF), (F32, F32), (F32, BF), (BF, F32)]
CANARY = 77.0


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    nv.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale + shift).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def within(got, ref, tol, what):
    got, tol = got.double(), torch.as_tensor(tol, dtype=torch.float64, device=got.device)
    bad = ~((got - ref).abs() <= tol) & ~((got == ref) | (got.isnan() & ref.isnan()))
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: got "
                             f"{got[i].item()!r}, {ref[i].item()!r} within {tol.expand_as(ref)[i].item():.3g}")


def placed(t, token_pad, head_pad, offset):
    """t (T, H, D) in a buffer of canaries: (buffer, view)."""
    T, H, D = t.shape
    hs = D + head_pad
    ts = H * hs + token_pad
    base = torch.full((offset + T * ts + 16,), CANARY, dtype=t.dtype, device="cuda")
    v = base.as_strided((T, H, D), (ts, hs, 1), offset)
    v.copy_(t)
    return base, v


def outside_untouched(base, view):
    """Every element of the buffer that is not the view's still holds the canary."""
    b = base.clone()
    b.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(CANARY)
    return bool((b == CANARY).all())


# ---------------------------------------------------------------- norm and rotation


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(R, dtype=torch.float64) / max(R, 1))).float().cuda()


def check_rope(x, y, pos, freq, gamma, eps, norm, inter, what):
    want, size = rope64(x, pos, freq, gamma, eps, norm, inter)
    within(y, want, U_OUT[y.dtype] * want.abs() + T_ROPE * size, what)


# tokens, query heads, key heads, values, pairs: each vector width, head size and number of lanes; odd ones
ROPE = [(1, 1, 1, 2, 1), (1, 40, 8, 128, 64), (3, 5, 1, 64, 32), (7, 3, 2, 96, 24), (5, 2, 2, 80, 40), (2, 3, 1, 10, 3),
        (33, 4, 4, 256, 128), (4, 2, 1, 512, 256), (9, 1, 3, 512, 1), (6, 2, 2, 96, 38), (5, 3, 1, 66, 0), (2, 1, 1, 130, 65),
        (2100, 2, 1, 64, 16), (2051, 1, 2, 34, 17), (4, 65, 3, 128, 54)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE)
def test_rope(T, Hq, Hk, D, R, xt, yt, inter):
    q, k = rand((T, Hq, D), xt, 1, 2.0), rand((T, Hk, D), xt, 2, 0.5, 0.3)
    gq, gk = rand((D,), F32, 3, 0.2, 1.0), rand((D,), F32, 4, 0.2, 1.0)
    pos, f = torch.randint(0, 5000, (T,), generator=gen(5), device="cuda", dtype=torch.int32), freqs(R)
    r = nv.nvfp4_qk_rope(q, k, pos, f, gq, gk, 1e-6, interleaved=inter, out_dtype=yt)
    assert r.q.dtype is yt and r.q.shape == q.shape and r.k.shape == k.shape
    check_rope(q, r.q, pos, f, gq, 1e-6, True, inter, "q")
    check_rope(k, r.k, pos, f, gk, 1e-6, True, inter, "k")
    r = nv.nvfp4_qk_rope(q, k, pos, f, norm=False, interleaved=inter, out_dtype=yt)
    check_rope(q, r.q, pos, f, None, 0, False, inter, "q turned")
    check_rope(k, r.k, pos, f, None, 0, False, inter, "k turned")


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("D,R,tp,hp,off", [(128, 64, 0, 0, 0), (128, 64, 8, 8, 8), (128, 64, 3, 0, 0), (64, 32, 4, 4, 4),
                                           (64, 32, 2, 2, 2), (96, 20, 0, 1, 1), (48, 24, 128, 0, 0)])
def test_rope_strides(D, R, tp, hp, off, xt, yt):
    """Heads that begin anywhere; nothing outside the results is written."""
    T, Hq, Hk = 9, 5, 2
    q, k = placed(rand((T, Hq, D), xt, 6), tp, hp, off)[1], placed(rand((T, Hk, D), xt, 7), tp, hp, off)[1]
    bq, oq = placed(torch.zeros((T, Hq, D), dtype=yt, device="cuda"), tp, hp, off)
    bk, ok = placed(torch.zeros((T, Hk, D), dtype=yt, device="cuda"), tp, hp, off)
    pos, f = torch.arange(T, device="cuda", dtype=torch.int32), freqs(R)
    g = rand((D,), BF, 8, 0.2, 1.0)
    r = nv.nvfp4_qk_rope(q, k, pos, f, g, g, 1e-5, out_q=oq, out_k=ok)
    assert r.q is oq and r.k is ok and outside_untouched(bq, oq) and outside_untouched(bk, ok)
    check_rope(q, oq, pos, f, g, 1e-5, True, False, "q")
    check_rope(k, ok, pos, f, g, 1e-5, True, False, "k")


def test_rope_packed_projection_and_in_place():
    """Queries and keys as parts of one product's rows, turned where they are; heads before tokens; weights for one only."""
    T, Hq, Hk, D = 37, 6, 2, 64
    packed = rand((T, (Hq + 2 * Hk) * D), BF, 9)
    heads = packed.view(T, Hq + 2 * Hk, D)
    q, k, v = heads[:, :Hq], heads[:, Hq:Hq + Hk], heads[:, Hq + Hk:].clone()
    pos, f, g = torch.arange(T, device="cuda", dtype=torch.int32) + 100, freqs(32), rand((D,), F32, 10, 0.1, 1.0)
    want = nv.nvfp4_qk_rope(q, k, pos, f, g, None)
    check_rope(q, want.q, pos, f, g, 1e-6, True, False, "q")
    check_rope(k, want.k, pos, f, None, 1e-6, True, False, "k")
    qh, kh = q.transpose(0, 1).contiguous().transpose(0, 1), k.transpose(0, 1).contiguous().transpose(0, 1)
    other = nv.nvfp4_qk_rope(qh, kh, pos, f, g, None)
    assert torch.equal(other.q, want.q) and torch.equal(other.k, want.k)
    nv.nvfp4_qk_rope(q, k, pos, f, g, None, out_q=q, out_k=k)
    assert torch.equal(q, want.q) and torch.equal(k, want.k) and torch.equal(heads[:, Hq + Hk:], v)


def test_rope_far_positions():
    """Angles keep their precision up to the last position."""
    pos = ints([0, 1, 4095, 131071, 10 ** 6 + 1, 16777217, 123456789, 2 ** 31 - 1, -5, -(2 ** 31)])
    f = freqs(32, 500000.0)
    x = rand((pos.numel(), 2, 64), F32, 11)
    r = nv.nvfp4_qk_rope(x, x, pos, f, norm=False)
    check_rope(x, r.q, pos, f, None, 0, False, False, "q")


def test_rope_odd_rows():
    """Zeros, a single large value, eps alone, and NaN that stays in its head."""
    x = rand((4, 3, 64), F32, 12)
    x[0, 0] = 0.0
    x[1, 1] = 0.0
    x[1, 1, 5] = 1e15
    x[2, 2] *= 1e-12
    pos, f = ints([0, 7, 70, 700]), freqs(16)
    clean = nv.nvfp4_qk_rope(x, x, pos, f)
    check_rope(x, clean.q, pos, f, None, 1e-6, True, False, "q")
    assert bool((clean.q[0, 0] == 0).all())
    y = x.clone()
    y[3, 1, 9] = float("nan")
    got = nv.nvfp4_qk_rope(y, y, pos, f).q
    assert bool(got[3, 1].isnan().all())
    got[3, 1] = clean.q[3, 1]
    assert torch.equal(got, clean.q)


def test_rope_empty():
    f, pos = freqs(16), ints([3, 4])
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")
    r = nv.nvfp4_qk_rope(z(0, 4, 64), z(0, 2, 64), ints([]), f)
    assert r.q.shape == (0, 4, 64)
    x = rand((2, 3, 64), BF, 13)
    r = nv.nvfp4_qk_rope(x, z(2, 0, 64), pos, f)
    check_rope(x, r.q, pos, f, None, 1e-6, True, False, "q")
    r = nv.nvfp4_qk_rope(z(2, 0, 64), x, pos, f)
    check_rope(x, r.k, pos, f, None, 1e-6, True, False, "k")
    g = nv.nvfp4_qk_rope_backward(z(0, 4, 64), z(0, 2, 64), z(0, 4, 64), z(0, 2, 64), ints([]), f)
    assert bool((g.dgamma_q == 0).all()) and bool((g.dgamma_k == 0).all())
    g = nv.nvfp4_qk_rope_backward(x, z(2, 0, 64), x, z(2, 0, 64), pos, f)
    assert bool((g.dgamma_k == 0).all()) and bool(g.dgamma_q.abs().sum() > 0)


def check_rope_grad(dy, x, dx, dg, pos, f, gamma, eps, norm, inter, what):
    want, size, wg, sg = rope_grad64(dy, x, pos, f, gamma, eps, norm, inter)
    within(dx, want, U_OUT[dx.dtype] * want.abs() + T_ROPE * size, "d" + what)
    if dg is not None:
        within(dg, wg, T_SUM * sg, "dgamma_" + what)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE)
def test_rope_backward(T, Hq, Hk, D, R, xt, yt, inter):
    q, k = rand((T, Hq, D), xt, 14, 2.0), rand((T, Hk, D), xt, 15, 0.5, 0.3)
    dq, dk = rand((T, Hq, D), yt, 16, 1e-3), rand((T, Hk, D), yt, 17, 1e-3)
    gq, gk = rand((D,), BF, 18, 0.2, 1.0), rand((D,), BF, 19, 0.2, 1.0)
    pos, f = torch.randint(0, 5000, (T,), generator=gen(20), device="cuda", dtype=torch.int32), freqs(R)
    r = nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, gq, gk, 1e-6, interleaved=inter)
    assert r.dq.dtype is xt and r.dgamma_q.shape == (D,)
    check_rope_grad(dq, q, r.dq, r.dgamma_q, pos, f, gq, 1e-6, True, inter, "q")
    check_rope_grad(dk, k, r.dk, r.dgamma_k, pos, f, gk, 1e-6, True, inter, "k")
    n = nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, gq, gk, 1e-6, interleaved=inter, want_dgamma=False)
    assert n.dgamma_q is None and torch.equal(n.dq, r.dq) and torch.equal(n.dk, r.dk)
    n = nv.nvfp4_qk_rope_backward(dq, dk, None, None, pos, f, norm=False, interleaved=inter)
    assert n.dgamma_q is None and n.dq.dtype is yt
    check_rope_grad(dq, None, n.dq, None, pos, f, None, 0, False, inter, "q turned back")


def test_rope_backward_is_deterministic_in_place_and_strided():
    T, Hq, Hk, D = 700, 5, 2, 64
    q, k = rand((T, Hq, D), BF, 21), rand((T, Hk, D), BF, 22)
    dq, dk = rand((T, Hq, D), BF, 23, 1e-3), rand((T, Hk, D), BF, 24, 1e-3)
    pos, f, g = torch.arange(T, device="cuda", dtype=torch.int32), freqs(32), rand((D,), F32, 25, 0.1, 1.0)
    a = nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, g, g)
    b = nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, g, g)
    for x, y in ((a.dq, b.dq), (a.dk, b.dk), (a.dgamma_q, b.dgamma_q), (a.dgamma_k, b.dgamma_k)):
        assert torch.equal(x, y)
    bq, oq = placed(torch.zeros_like(q), 3, 1, 1)
    bk, ok = placed(torch.zeros_like(k), 3, 1, 1)
    nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, g, g, out_q=oq, out_k=ok)
    assert outside_untouched(bq, oq) and outside_untouched(bk, ok)
    check_rope_grad(dq, q, oq, None, pos, f, g, 1e-6, True, False, "q")
    dq2, dk2, q2, k2 = dq.clone(), dk.clone(), q.clone(), k.clone()
    nv.nvfp4_qk_rope_backward(dq2, dk2, q, k, pos, f, g, g, out_q=dq2, out_k=dk2)
    nv.nvfp4_qk_rope_backward(dq, dk, q2, k2, pos, f, g, g, out_q=q2, out_k=k2)
    assert torch.equal(dq2, a.dq) and torch.equal(dk2, a.dk) and torch.equal(q2, a.dq) and torch.equal(k2, a.dk)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_backward_against_differences(inter):
    """Central differences of the 64-bit forward pass along random directions."""
    T, Hq, Hk, D, R = 3, 2, 1, 32, 12
    q, k = rand((T, Hq, D), F32, 26), rand((T, Hk, D), F32, 27)
    dq, dk = rand((T, Hq, D), F32, 28), rand((T, Hk, D), F32, 29)
    gq, gk = rand((D,), F32, 30, 0.2, 1.0), rand((D,), F32, 31, 0.2, 1.0)
    pos, f = ints([0, 5, 900]), freqs(R)
    r = nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, gq, gk, 1e-4, interleaved=inter)

    def loss(q, k, gq, gk):
        a = rope64(q, pos, f, gq, 1e-4, True, inter)[0]
        b = rope64(k, pos, f, gk, 1e-4, True, inter)[0]
        return float((a * dq.double()).sum() + (b * dk.double()).sum())
    args, grads = [t.double() for t in (q, k, gq, gk)], (r.dq, r.dk, r.dgamma_q, r.dgamma_k)
    h = 1e-5
    for i in range(4):
        for seed in range(3):
            d = rand(args[i].shape, F32, 32 + seed).double()
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * d, args[i] - h * d
            slope = (loss(*up) - loss(*down)) / (2 * h)
            got = float((grads[i].double() * d).sum())
            bar = 1e-4 * float((grads[i].double() * d).abs().sum())  # fp32 gradient, h^2 of the third derivative
            assert abs(got - slope) <= bar + 1e-7, (i, seed, got, slope)


# ---------------------------------------------------------------- the cache


class Work:
    """A batch on pages in a shuffled order, with spare pages around."""

    def __init__(self, lens, news, heads, dim, page, alpha=(2.0 ** -5, 2.0 ** -6), seed=0, behind=0, order="phsd"):
        self.lens, self.news, self.page = lens, news, page
        used = [-(-n // page) for n in lens]
        P = sum(used) + 2
        perm = torch.randperm(P, generator=gen(seed + 1), device="cuda").to(torch.int32)
        W = max(used + [1])
        self.table = torch.full((len(lens), W), -1, dtype=torch.int32, device="cuda")  # beyond a sequence: nothing
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = perm[at:at + n]
            at += n
        starts = [0]
        for m in news:
            starts.append(starts[-1] + m)
        self.T = starts[-1] + behind
        self.starts, self.lengths = ints(starts), ints(lens)

        def space(n, top):  # NaN scales wherever nothing is written
            shape = {"phsd": (P, heads, page, n), "pshd": (P, page, heads, n), "hpsd": (heads, P, page, n)}[order]
            t = torch.full(shape, top, dtype=torch.uint8, device="cuda")
            return {"phsd": t, "pshd": t.permute(0, 2, 1, 3), "hpsd": t.permute(1, 0, 2, 3)}[order]
        self.cache = nv.KVCache(space(dim // 2, 0x73), space(dim // 16, 0x7F), space(dim // 2, 0x73),
                                space(dim // 16, 0x7F), torch.tensor(alpha, dtype=F32, device="cuda"))
        self.heads, self.dim, self.seed = heads, dim, seed

    @property
    def batch(self):
        return self.starts, self.lengths, self.table

    def fill(self, dtype=BF, scale=1.0):
        """Every token of every sequence written at once; returns the keys and values."""
        lens = self.lens
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        k = rand((starts[-1], self.heads, self.dim), dtype, self.seed + 2, scale)
        v = rand((starts[-1], self.heads, self.dim), dtype, self.seed + 3, scale)
        st = ints([0])
        nv.nvfp4_cache_write(k, v, self.cache, ints(starts), self.lengths, self.table, status=st)
        assert st.item() == 0
        return k, v

    def slots(self):
        """(page, row) of each row of the call."""
        out = []
        t = self.table.tolist()
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            out += [(t[b][j // self.page], j % self.page) for j in range(n - m, n)]
        return out


def packed(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def check_written(w, k, v):
    pages, rows = (torch.tensor(x) for x in zip(*w.slots()))
    for x, c, s, a in ((k, w.cache.k_codes, w.cache.k_scales, 0), (v, w.cache.v_codes, w.cache.v_scales, 1)):
        codes, scales = quantize32(x[:pages.numel()], w.cache.alpha[a].item())
        assert torch.equal(s.cpu()[pages, :, rows].view(torch.float8_e4m3fn).float(), scales)
        got = c.cpu()[pages, :, rows]
        low, high = got & 15, got >> 4
        got = torch.stack([low, high], -1).flatten(-2).long()
        got = torch.where(got == 8, torch.zeros_like(got), got)  # -0 is 0
        codes = torch.where(codes == 8, torch.zeros_like(codes), codes)
        assert torch.equal(got, codes)


CACHE = [([1], [1], 1, 32, 16), ([5, 17, 0, 33], [1, 1, 0, 1], 2, 64, 16), ([40, 7], [40, 7], 3, 96, 48),
         ([100], [37], 1, 256, 32), ([64, 64, 1], [64, 3, 1], 8, 128, 64), ([33, 2, 90], [30, 2, 0], 5, 160, 80)]


@pytest.mark.parametrize("order", ["phsd", "pshd", "hpsd"])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("lens,news,heads,dim,page", CACHE)
def test_cache_write_and_read(lens, news, heads, dim, page, xt, order):
    w = Work(lens, news, heads, dim, page, seed=40, behind=3, order=order)
    k, v = rand((w.T, heads, dim), xt, 41, 3.0), rand((w.T, heads, dim), xt, 42, 0.01)
    before = [t.clone() for t in w.cache.tensors()]
    st = ints([0])
    nv.nvfp4_cache_write(k, v, w.cache, *w.batch, status=st)
    assert st.item() == 0
    check_written(w, k, v)
    written = torch.zeros(w.cache.k_codes.shape[:3], dtype=torch.bool)
    for p, r in w.slots():
        written[p, :, r] = True
    for t, b in zip(w.cache.tensors()[:4], before):  # nothing else
        assert torch.equal(t.cpu()[~written], b.cpu()[~written])
    for yt in (BF, F32):
        out = torch.full((w.T, heads, dim), CANARY, dtype=yt, device="cuda")
        r = nv.nvfp4_cache_read(w.cache, *w.batch, out_k=out, out_v=out.clone(), status=st)
        n = sum(news)
        for i, (x, got) in enumerate(((k, r.k), (v, r.v))):
            codes, scales = quantize32(x[:n], w.cache.alpha[i].item())
            grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6])
            val = torch.cat([grid, -grid])[codes] * scales.repeat_interleave(16, -1) * w.cache.alpha[i].item()
            assert torch.equal(got[:n].cpu(), val.to(yt)) and bool((got[n:] == CANARY).all())
    assert st.item() == 0


@pytest.mark.parametrize("alpha", [(1.0, 2.0 ** -10), (0.0123, 3.7e-4), (2.0 ** 20, 1e-12), (2.0 ** -100, 2.0 ** 100)])
def test_cache_write_any_tensor_scale(alpha):
    """Scales that saturate and that vanish, values on the middles of two codes."""
    w = Work([50], [50], 2, 64, 16, alpha, seed=43)
    k, v = rand((50, 2, 64), F32, 44, alpha[0] * 10), rand((50, 2, 64), F32, 45, alpha[1] * 300)
    k[0] = 0.0
    k[1] = k[1] * 1e-3
    k[2] = k[2] * 1e-5
    k[3] = k[3] * 1e4
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda").repeat(8) * alpha[0]
    for i in range(40):
        k[10 + i, 0] = mids * (2.0 ** (i % 5)) * (1 + (i % 8) / 8)
    nv.nvfp4_cache_write(k, v, w.cache, *w.batch)
    check_written(w, k, v)


def test_cache_write_matches_the_quantizer():
    """Where alpha is a power of two and no value is next to a middle, the bytes are nvfp4_quantize's."""
    w = Work([128], [128], 2, 128, 64, (1.0 / 64, 1.0 / 64), seed=46)
    k, v = rand((128, 2, 128), BF, 47), rand((128, 2, 128), BF, 48)
    nv.nvfp4_cache_write(k, v, w.cache, *w.batch)
    amax = torch.full((2,), 2688.0 / 64, device="cuda")
    q = nv.nvfp4_quantize(k.view(256, 128), amax, nv.ROWWISE)
    pages, rows = (torch.tensor(x, device="cuda") for x in zip(*w.slots()))
    s = w.cache.k_scales[pages, :, rows].reshape(256, 8)
    c = w.cache.k_codes[pages, :, rows].reshape(256, 64)
    assert torch.equal(s, q.s_row)
    assert float((c != q.q_row).float().mean()) < 0.03  # ties through the rounded reciprocal


def test_cache_write_nonfinite_and_bad_alpha():
    w = Work([20], [20], 1, 32, 16, seed=49)
    k, v = rand((20, 1, 32), F32, 50), rand((20, 1, 32), F32, 51)
    k[3, 0, 5], k[4, 0, 20], v[7, 0, 0] = float("nan"), float("inf"), float("-inf")
    st = ints([0])
    nv.nvfp4_cache_write(k, v, w.cache, *w.batch, status=st)
    assert st.item() == -6
    check_written(w, k, v)
    r = nv.nvfp4_cache_read(w.cache, *w.batch, tokens=20, out_dtype=F32)
    assert bool(r.k.isfinite().all()) and r.k[3, 0, 5] == 0 and r.k[4, 0, 20] == 2688 * 2.0 ** -5
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 101):
        before = w.cache.k_codes.clone()
        w.cache.alpha[1] = bad
        st.zero_()
        nv.nvfp4_cache_write(v, k, w.cache, *w.batch, status=st)
        assert st.item() == -7 and torch.equal(before, w.cache.k_codes)


def test_cache_bad_numbers_are_left_out():
    """Pages, lengths and starts out of range: their tokens are left out, the others are right, status says so."""
    lens, news = [30, 40, 20], [4, 40, 6]
    w = Work(lens, news, 2, 32, 16, seed=52)
    k, v = rand((w.T, 2, 32), BF, 53), rand((w.T, 2, 32), BF, 54)
    nv.nvfp4_cache_write(k, v, w.cache, *w.batch)
    good = nv.nvfp4_cache_read(w.cache, *w.batch, tokens=w.T)
    P = w.cache.k_codes.shape[0]
    for bad in (-1, P, 2 ** 31 - 1, -(2 ** 31)):
        t = w.table.clone()
        t[1, 1] = bad  # positions 16..31 of the second sequence: rows 4 + 16 ..
        st = ints([0])
        out = torch.full((w.T, 2, 32), CANARY, dtype=BF, device="cuda")
        r = nv.nvfp4_cache_read(w.cache, w.starts, w.lengths, t, out_k=out, want_v=False, status=st)
        assert st.item() == -9 and r.v is None
        assert bool((out[20:36] == 0).all())
        assert torch.equal(out[:20], good.k[:20]) and torch.equal(out[36:], good.k[36:])
        before = [x.clone() for x in w.cache.tensors()]
        st.zero_()
        nv.nvfp4_cache_write(k, v, w.cache, w.starts, w.lengths, t, status=st)
        assert st.item() == -9
        assert all(torch.equal(a, b) for a, b in zip(before, w.cache.tensors()))
    for starts, lengths, left in (([0, 4, 44, 50], [30, 49, 20], range(4, 44)), ([0, 4, 44, 50], [30, -1, 20], range(4, 44)),
                                  ([0, 4, 44, 51], [30, 40, 20], range(44, 50)), ([-1, 4, 44, 50], [30, 40, 20], range(0, 4))):
        st = ints([0])
        out = torch.full((w.T, 2, 32), CANARY, dtype=BF, device="cuda")
        nv.nvfp4_cache_read(w.cache, ints(starts), ints(lengths), w.table, out_k=out, want_v=False, status=st)
        assert st.item() == -9
        rows = torch.zeros(w.T, dtype=torch.bool)
        rows[list(left)] = True
        assert bool((out[rows] == CANARY).all()) and torch.equal(out[~rows], good.k[~rows])
    st = ints([0])  # more new tokens than there are: negative positions
    out = torch.full((w.T, 2, 32), CANARY, dtype=BF, device="cuda")
    nv.nvfp4_cache_read(w.cache, w.starts, ints([2, 40, 20]), w.table, out_k=out, want_v=False, status=st)
    assert st.item() == -9 and bool((out[:2] == 0).all()) and torch.equal(out[4:], good.k[4:])


# ---------------------------------------------------------------- attention


def check_attention(w, q, r, scale=None, causal=True, window=0, sinks=0, table=None):
    t = w.table if table is None else table
    o, lse, size, score = attend64(q, w.cache, w.starts, w.lengths, t, scale, causal, window, sinks)
    n = w.starts[-1].item()
    d = (T_SCORE * score)[:n]
    within(r.o[:n], o[:n], U_OUT[BF] * o[:n].abs() + (T_WEIGHT + 2 * d[..., None]) * size[:n], "o")
    if r.lse is not None:
        within(r.lse[:n], lse[:n], d + 2.0 ** -17 + 2.0 ** -23 * lse[:n].abs().nan_to_num(0.0, posinf=0.0), "lse")


def attend(w, Hq, seed=60, scale=1.0, **kw):
    q = rand((w.T, Hq, w.dim), BF, seed, scale)
    st = ints([0])
    r = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True, status=st, **kw)
    assert st.item() == 0
    check_attention(w, q, r, **kw)
    return q, r


def among_rows(t, T):
    """t (tokens, heads, values) as the first of T tokens, its strides (where tokens or heads come first) and the alignment
    of its address kept."""
    n, H, D = t.shape
    ts, hs = (t.stride(0) if n > 1 else H * D), (t.stride(1) if H > 1 else D)
    if H > 1 and n > 1 and hs > ts:
        hs = T * ts
    off = t.data_ptr() % 16 // t.element_size()
    base = torch.zeros(off + (T - 1) * ts + (H - 1) * hs + D, dtype=t.dtype, device="cuda")
    v = base.as_strided((T, H, D), (ts, hs, 1), off)
    v[:n] = t
    return v


@pytest.fixture(params=["alone", "crowded"])
def company(request, monkeypatch):
    """Which kernel takes a sequence depends on the whole batch (few hundred tiles of 16 rows over all key heads are few):
    each call as it is, and with so many rows behind the last sequence and so many empty ones that sequences of more than
    32 rows to a key head go to the kernel for many."""
    call = nv.nvfp4_cache_attention

    def crowded(q, cache, starts, lengths, pages, *args, out=None, **kw):
        n, heads, B = q.shape[0], cache.k_codes.shape[1], lengths.shape[0]
        more = 183 // heads + 1
        T = n + B + more + 366 * 16 * heads // q.shape[1] + 1
        starts = torch.cat([starts, starts[-1:].expand(more)])
        lengths = torch.cat([lengths, lengths.new_zeros(more)])
        pages = torch.cat([pages, pages.new_zeros(more, pages.shape[1])])
        rows = among_rows(q, T)
        o = among_rows(out, T) if out is not None and out is not q else rows if out is q else None
        r = call(rows, cache, starts, lengths, pages, *args, out=o, **kw)
        if out is not None:
            out.copy_(r.o[:n])
        return nv.AttentionOut(out if out is not None else r.o[:n], None if r.lse is None else r.lse[:n])

    if request.param == "crowded":
        monkeypatch.setattr(nv, "nvfp4_cache_attention", crowded)


both_kernels = pytest.mark.usefixtures("company")


# lengths, new tokens, key heads, queries to each, dim, page
ATTEND = [([1], [1], 1, 1, 32, 16), ([17], [1], 2, 5, 128, 16), ([700], [1], 8, 5, 128, 16), ([64, 65, 63, 1], [1] * 4, 2, 8, 64, 32),
          ([300, 5, 0, 999], [1, 1, 0, 1], 3, 7, 96, 48), ([513], [1], 1, 16, 256, 64), ([90, 200], [1, 1], 1, 20, 160, 16),
          ([130, 77], [4, 3], 2, 5, 128, 32), ([40, 40], [40, 17], 2, 3, 64, 16), ([257], [129], 1, 4, 128, 64),
          ([333, 48, 2], [300, 1, 2], 2, 1, 96, 16), ([200], [50], 1, 8, 224, 48), ([150], [150], 1, 2, 192, 16),
          ([260, 129], [257, 128], 1, 2, 256, 128), ([5000], [2], 1, 3, 64, 64), ([30] * 70, [1] * 70, 2, 2, 32, 16)]


@both_kernels
@pytest.mark.parametrize("lens,news,heads,group,dim,page", ATTEND)
def test_attention(lens, news, heads, group, dim, page):
    w = Work(lens, news, heads, dim, page, seed=61, behind=2)
    w.fill()
    q = rand((w.T, heads * group, dim), BF, 62)
    out = torch.full_like(q, CANARY)
    st = ints([0])
    r = nv.nvfp4_cache_attention(q, w.cache, *w.batch, out=out, want_lse=True, status=st)
    assert st.item() == 0 and r.o is out
    check_attention(w, q, r)
    assert bool((out[w.T - 2:] == CANARY).all())  # rows behind the last sequence
    attend(w, heads * group, causal=False)
    attend(w, heads * group, scale=0.3)


@both_kernels
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 4), (37, 17), (128, 1000), (10 ** 6, 3), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("lens,news,heads,group,dim,page", [
    ([500, 3, 170], [1, 1, 1], 2, 5, 128, 16), ([300, 64], [4, 9], 1, 8, 64, 48), ([270, 130], [200, 130], 2, 2, 96, 32),
    ([400], [333], 1, 3, 256, 64)])
def test_attention_window_and_sinks(lens, news, heads, group, dim, page, window, sinks):
    w = Work(lens, news, heads, dim, page, seed=63)
    w.fill()
    attend(w, heads * group, window=window, sinks=sinks)


@both_kernels
def test_attention_rows_that_see_nothing():
    """More new tokens than the sequence holds: the first rows lie before its beginning; lengths of zero."""
    for lens, news in (([3, 0, 40], [5, 2, 41]), ([0], [1]), ([2], [300]), ([0, 0], [200, 1])):
        w = Work(lens, [0] * len(lens), 2, 64, 16, seed=64)
        w.fill()
        w.news = news
        starts = [0]
        for m in news:
            starts.append(starts[-1] + m)
        w.starts, w.T = ints(starts), starts[-1]
        q, r = attend(w, 4)
        for b, (n, m) in enumerate(zip(lens, news)):
            first = r.o[starts[b]:starts[b] + max(0, m - n)]
            assert bool((first == 0).all()) and bool((r.lse[starts[b]:starts[b] + max(0, m - n)] == -math.inf).all())
        attend(w, 4, causal=False)


@both_kernels
@pytest.mark.parametrize("news", [[1, 1, 1], [6, 1, 30], [150, 90, 200]])
def test_attention_ignores_what_it_must_not_see(news):
    """Bytes behind a sequence's end, in other pages and in later tokens change no row that does not see them."""
    lens = [150, 90, 210]
    w = Work(lens, news, 2, 128, 32, seed=65)
    k, v = w.fill()
    q, r = attend(w, 10)
    c = w.cache
    nan, codes = c.k_scales == 0x7F, c.k_codes.clone()
    for t in (c.k_scales, c.v_scales):
        t[nan] = 0xFF  # other NaNs, beyond every length
    again = nv.nvfp4_cache_attention(q, c, *w.batch, want_lse=True)
    assert torch.equal(again.o, r.o) and torch.equal(again.lse, r.lse)
    assert torch.equal(codes, c.k_codes)
    # the last token of each sequence becomes huge: only its own row changes
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    last = torch.zeros(sum(news), dtype=torch.bool)
    for b in range(3):
        k[starts[b + 1] - 1] = 1e30
        v[starts[b + 1] - 1] = float("inf")
    nv.nvfp4_cache_write(k, v, c, ints(starts), w.lengths, w.table)
    at = 0
    for m in news:
        at += m
        last[at - 1] = True
    other = nv.nvfp4_cache_attention(q, c, *w.batch, want_lse=True)
    assert torch.equal(other.o[~last], r.o[~last]) and torch.equal(other.lse[~last], r.lse[~last])
    check_attention(w, q, other)


@both_kernels
@pytest.mark.parametrize("news", [[1, 1], [9, 30], [150, 180]])
def test_attention_odd_queries(news):
    """Large and tiny queries, zeros, and NaN and Inf that stay in their rows."""
    w = Work([150, 200], news, 1, 64, 16, seed=66)
    w.fill()
    q = rand((w.T, 3, 64), BF, 67)
    q[0, 0] *= 100.0
    q[0, 1] = 0.0
    q[0, 2] *= 2.0 ** -40
    q[1, 0, 3] = 3e4
    q[1, 1, :32] *= 2.0 ** -20
    r = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True)
    check_attention(w, q, r)
    bad = q.clone()
    bad[1, 2, 7] = float("nan")
    bad[0, 1, 9] = float("inf")
    got = nv.nvfp4_cache_attention(bad, w.cache, *w.batch, want_lse=True)
    assert bool(got.o[1, 2].isnan().all()) and bool(got.lse[1, 2].isnan())
    keep = torch.ones((w.T, 3), dtype=torch.bool)
    keep[1, 2] = keep[0, 1] = False
    assert torch.equal(got.o[keep], r.o[keep]) and torch.equal(got.lse[keep], r.lse[keep])


@both_kernels
@pytest.mark.parametrize("news", [[1, 1, 1], [8, 1, 100]])
def test_attention_rising_and_falling_scores(news):
    """Scores that climb over the whole sequence (the running maximum moves all the time) and that fall."""
    lens = [600, 333, 400]
    for sign in (1.0, -1.0):
        w = Work(lens, news, 1, 64, 16, (2.0 ** -4, 2.0 ** -6), seed=68)
        k = torch.cat([torch.linspace(-1, 1, n, device="cuda") for n in lens])[:, None, None] * sign * torch.ones((1, 1, 64), device="cuda") * 3
        v = rand((sum(lens), 1, 64), BF, 69)
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        nv.nvfp4_cache_write(k.to(BF), v, w.cache, ints(starts), w.lengths, w.table)
        q = (torch.ones((w.T, 5, 64), device="cuda") * torch.tensor([0.1, 1, 4, -2, 0.5], device="cuda")[None, :, None]).to(BF)
        r = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True)
        check_attention(w, q, r)


@both_kernels
@pytest.mark.parametrize("order", ["pshd", "hpsd"])
@pytest.mark.parametrize("news", [[1, 1], [5, 140]])
def test_attention_layouts(order, news):
    """Caches in other orders, queries and results with odd strides and bases; in place."""
    w = Work([140, 190], news, 2, 96, 16, seed=70, order=order)
    w.fill()
    q0 = rand((w.T, 6, 96), BF, 71)
    want = nv.nvfp4_cache_attention(q0, w.cache, *w.batch).o
    for tp, hp, off in ((0, 0, 1), (8, 8, 8), (3, 1, 5), (64, 0, 0)):
        q = placed(q0, tp, hp, off)[1]
        base, out = placed(torch.zeros_like(q0), tp, hp, off)
        r = nv.nvfp4_cache_attention(q, w.cache, *w.batch, out=out, want_lse=True)
        check_attention(w, q, r)
        assert torch.equal(out, want) and outside_untouched(base, out)
    heads_first = q0.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(nv.nvfp4_cache_attention(heads_first, w.cache, *w.batch).o, want)
    q = q0.clone()
    nv.nvfp4_cache_attention(q, w.cache, *w.batch, out=q)
    assert torch.equal(q, want)


@both_kernels
@pytest.mark.parametrize("news", [[1, 1, 1], [4, 170, 1]])
def test_attention_bad_pages(news):
    """Pages out of range hide their tokens; sequences with bad numbers keep their rows as they were."""
    w = Work([100, 200, 50], news, 2, 64, 16, seed=72)
    w.fill()
    q = rand((w.T, 4, 64), BF, 73)
    t = w.table.clone()
    t[0, 2], t[1, 0], t[1, 7], t[2, 0] = -1, w.cache.k_codes.shape[0], 2 ** 31 - 1, -(2 ** 31)
    st = ints([0])
    r = nv.nvfp4_cache_attention(q, w.cache, w.starts, w.lengths, t, want_lse=True, status=st)
    assert st.item() == -9
    check_attention(w, q, r, table=t)
    good = nv.nvfp4_cache_attention(q, w.cache, *w.batch).o
    for lengths in ([100, -3, 50], [100, 10 ** 6, 50]):
        out = torch.full_like(q, CANARY)
        st.zero_()
        nv.nvfp4_cache_attention(q, w.cache, w.starts, ints(lengths), w.table, out=out, status=st)
        a, b = w.starts[1].item(), w.starts[2].item()
        assert st.item() == -9 and bool((out[a:b] == CANARY).all())
        assert torch.equal(out[:a], good[:a]) and torch.equal(out[b:], good[b:])


def test_attention_two_sequences_share_pages():
    """A common beginning on shared pages, as for several answers to one prompt."""
    w = Work([100, 100, 100], [1, 1, 1], 2, 64, 16, seed=74)
    w.table[1, :4] = w.table[0, :4]
    w.table[2] = w.table[0]
    w.cache.k_scales.fill_(0x40)
    w.cache.v_scales.fill_(0x38)
    for c in (w.cache.k_codes, w.cache.v_codes):
        c.copy_(torch.randint(0, 256, c.shape, generator=gen(75), device="cuda", dtype=torch.uint8))
    attend(w, 6, scale=0.01)


def test_attention_same_bits_every_time_and_with_other_company():
    """The same call gives the same bits; a captured one, replayed with new lengths, too."""
    w = Work([800, 90, 1500], [1, 1, 1], 2, 128, 32, seed=76)
    w.fill()
    q, r = attend(w, 10)
    for _ in range(3):
        again = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True)
        assert torch.equal(again.o, r.o) and torch.equal(again.lse, r.lse)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        nv.nvfp4_cache_attention(q, w.cache, *w.batch, out=out)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        nv.nvfp4_cache_attention(q, w.cache, *w.batch, out=out)
    for lens in ([800, 90, 1500], [33, 90, 1400], [0, 1, 700]):
        w.lengths.copy_(ints(lens))
        g.replay()
        assert torch.equal(out, nv.nvfp4_cache_attention(q, w.cache, *w.batch).o)
        check_attention(w, q, nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True))


def test_on_another_stream():
    w = Work([300, 20], [1, 1], 2, 64, 16, seed=77)
    s = torch.cuda.Stream()
    k, v, q = rand((2, 2, 64), BF, 78), rand((2, 2, 64), BF, 79), rand((2, 4, 64), BF, 80)
    w.fill()
    pos, f = ints([299, 19]), freqs(32)
    torch.cuda.synchronize()
    a = nv.nvfp4_qk_rope(q, k, pos, f, stream=s)
    nv.nvfp4_cache_write(a.k, v, w.cache, *w.batch, stream=s)
    r = nv.nvfp4_cache_attention(a.q, w.cache, *w.batch, want_lse=True, stream=s.cuda_stream)
    c = nv.nvfp4_cache_read(w.cache, *w.batch, tokens=2, stream=s)
    b = nv.nvfp4_qk_rope_backward(r.o, c.k, q, k, pos, f, stream=s)
    s.synchronize()
    check_attention(w, a.q, r)
    check_rope_grad(r.o, q, b.dq, b.dgamma_q, pos, f, None, 1e-6, True, False, "q")


def test_refusals():
    w = Work([30], [1], 2, 64, 16, seed=81)
    w.fill()
    q, k = rand((1, 4, 64), BF, 82), rand((1, 2, 64), BF, 83)
    att = lambda q=q, cache=w.cache, batch=w.batch, **kw: nv.nvfp4_cache_attention(q, cache, *batch, **kw)
    for bad in (q.float(), q.half()):
        with pytest.raises(TypeError):
            att(bad)
    with pytest.raises(TypeError):
        att(q[0])
    with pytest.raises(ValueError):
        att(rand((1, 4, 96), BF, 84))
    with pytest.raises(nv.Nvfp4Error):
        att(rand((1, 3, 64), BF, 85))  # no multiple of the key heads
    with pytest.raises(ValueError):
        att(q.cpu())
    for kw in (dict(window=-1), dict(sinks=2), dict(window=4, causal=False), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=8, sinks=-1), dict(window=2 ** 31)):
        with pytest.raises(nv.Nvfp4Error):
            att(**kw)
    with pytest.raises(TypeError):
        att(batch=(w.starts.long(), w.lengths, w.table))
    with pytest.raises(ValueError):
        att(batch=(w.starts[:1], w.lengths, w.table))
    with pytest.raises(ValueError):
        att(batch=(w.starts, w.lengths, w.table.repeat(2, 1)))
    with pytest.raises(TypeError):
        att(batch=(w.starts, w.lengths, w.table.float()))
    with pytest.raises(ValueError):
        att(out=torch.empty_like(q).expand(1, 4, 64)[:, :1].expand(1, 4, 64))
    c = w.cache
    for bad, err in ((nv.KVCache(c.k_codes.float(), *c.tensors()[1:]), TypeError),
                     (nv.KVCache(c.k_codes, c.k_scales[..., :2], *c.tensors()[2:]), ValueError),
                     (nv.KVCache(c.k_codes, c.k_scales, c.v_codes.transpose(0, 1).contiguous().transpose(0, 1),
                                 c.v_scales, c.alpha), ValueError),
                     (nv.KVCache(*c.tensors()[:4], c.alpha[:1]), ValueError),
                     (nv.KVCache(*c.tensors()[:4], c.alpha.double()), TypeError),
                     (nv.KVCache(*(t[:, :, :8] for t in c.tensors()[:4]), c.alpha), nv.Nvfp4Error)):  # pages of 8
        with pytest.raises(err):
            att(cache=bad)
    with pytest.raises(ValueError):
        nv.nvfp4_cache_write(k, k[:, :1], c, *w.batch)
    with pytest.raises(TypeError):
        nv.nvfp4_cache_write(k, k.float(), c, *w.batch)
    with pytest.raises(TypeError):
        nv.nvfp4_cache_read(c, *w.batch)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_cache_read(c, *w.batch, tokens=-1)
    pos, f = ints([3]), freqs(32)
    rope = lambda **kw: nv.nvfp4_qk_rope(**{**dict(q=q, k=k, positions=pos, inv_freq=f), **kw})
    for kw, err in ((dict(positions=pos.long()), TypeError), (dict(positions=ints([1, 2])), ValueError),
                    (dict(inv_freq=freqs(33)), nv.Nvfp4Error), (dict(inv_freq=f.double()), TypeError),
                    (dict(k=k[..., :32]), ValueError), (dict(k=k.float()), TypeError), (dict(q=q.half()), TypeError),
                    (dict(gamma_q=torch.ones(32, device="cuda")), ValueError),
                    (dict(gamma_q=torch.ones(64, device="cuda"), norm=False), nv.Nvfp4Error),
                    (dict(gamma_q=torch.ones(64, device="cuda"), gamma_k=torch.ones(64, device="cuda", dtype=BF)), TypeError),
                    (dict(eps=-1.0), nv.Nvfp4Error), (dict(eps=float("nan")), nv.Nvfp4Error),
                    (dict(out_dtype=torch.float16), TypeError), (dict(out_q=q.float(), out_dtype=BF), TypeError)):
        with pytest.raises(err):
            rope(**kw)
    with pytest.raises(TypeError):
        nv.nvfp4_qk_rope_backward(q, k, None, None, pos, f)


def test_empty_batches():
    w = Work([30], [1], 2, 64, 16, seed=86)
    w.fill()
    z = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    assert nv.nvfp4_cache_attention(z, w.cache, ints([0, 0]), w.lengths, w.table, want_lse=True).o.shape == (0, 4, 64)
    none = (ints([0]), ints([]), torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    out = torch.full((2, 4, 64), CANARY, dtype=BF, device="cuda")
    nv.nvfp4_cache_attention(rand((2, 4, 64), BF, 87), w.cache, *none, out=out)
    assert bool((out == CANARY).all())
    nv.nvfp4_cache_write(z[:, :2], z[:, :2], w.cache, ints([0, 0]), w.lengths, w.table)
    assert nv.nvfp4_cache_read(w.cache, *none, tokens=0).k.shape == (0, 2, 64)
    # sequences without pages at all
    st = ints([0])
    out = torch.full((2, 4, 64), CANARY, dtype=BF, device="cuda")
    r = nv.nvfp4_cache_attention(rand((2, 4, 64), BF, 88), w.cache, ints([0, 2]), ints([0]),
                                 torch.empty((1, 0), dtype=torch.int32, device="cuda"), out=out, want_lse=True, status=st)
    assert st.item() == 0 and bool((out == 0).all()) and bool((r.lse == -math.inf).all())


# ---------------------------------------------------------------- together, and around the calls


def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_an_attention_block(window, sinks):
    """The example: prompts and then tokens one at a time.  Each NVFP4 operand is off by about 0.1 of its norm, so a
    product by 0.14; two products and the cached values in a row: 0.25."""
    far = example().run(640, 10, 2, [150, 33, 70], dim=64, window=window, sinks=sinks)
    assert all(v <= 0.35 for v in far.values()), far


@both_kernels
def test_the_calls_together_match_the_formulas():
    """Rotation, write and attention as a decoder makes them, for a prompt and the tokens behind it, against the
    formulas on what the calls before left."""
    Hq, Hk, D, page = 6, 2, 96, 48
    f, g = freqs(48), rand((D,), F32, 90, 0.1, 1.0)
    pages = ints([[3, 0, 2, 5]])
    cache = nv.nvfp4_kv_cache(6, Hk, page, D, (2.0 ** -5, 2.0 ** -5))
    length = 0
    for n in (130, 1, 1, 7, 40):
        qkv = rand((n, Hq + 2 * Hk, D), BF, 91 + n)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        pos = torch.arange(length, length + n, device="cuda", dtype=torch.int32)
        length += n
        q0, k0 = q.clone(), k.clone()
        r = nv.nvfp4_qk_rope(q, k, pos, f, g, g, out_q=q, out_k=k)
        check_rope(q0, r.q, pos, f, g, 1e-6, True, False, "q")
        check_rope(k0, r.k, pos, f, g, 1e-6, True, False, "k")
        batch = (ints([0, n]), ints([length]), pages)
        nv.nvfp4_cache_write(r.k, v, cache, *batch)
        c = nv.nvfp4_cache_read(cache, *batch, tokens=n, out_dtype=F32)
        for x, y in ((r.k, c.k), (v, c.v)):  # half a step of E2M1 at most, of the block's largest value / 6
            top = x.float().unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
            assert bool(((x.float() - y).abs() <= top * (1 / 6 + 2.0 ** -4) + 1e-3).all())
        o = nv.nvfp4_cache_attention(r.q, cache, *batch, want_lse=True)
        w = type("W", (), dict(cache=cache, starts=batch[0], lengths=batch[1], table=pages))()
        check_attention(w, r.q, o)


def test_workspaces_are_not_overrun():
    """Guard bytes around a workspace of exactly the size that the C ABI asks for, for one and many rows."""
    import ctypes
    from nvfp4_bit_block_gb300.attention import Batch, Cache, Tokens
    L = nv.attention_lib()
    for news, dim, group in (([1, 1, 1], 64, 5), ([3, 1, 1], 128, 5), ([1, 1, 1], 256, 2), ([2, 30, 90], 128, 4), ([1, 1, 1], 96, 20)):
        w = Work([700, 90, 333], news, 2, dim, 16, seed=92)
        w.fill()
        Hq = 2 * group
        q = rand((w.T, Hq, dim), BF, 93)
        want = nv.nvfp4_cache_attention(q, w.cache, *w.batch).o
        n = L.nvfp4_cache_attention_workspace(w.T, Hq, 2, dim, 3)
        ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        o = torch.empty_like(q)
        c, kc, sc = w.cache, w.cache.k_codes, w.cache.k_scales
        cache = Cache(c.k_codes.data_ptr(), c.k_scales.data_ptr(), c.v_codes.data_ptr(), c.v_scales.data_ptr(),
                      c.alpha.data_ptr(), kc.shape[0], 2, 16, dim, *kc.stride()[:3], *sc.stride()[:3])
        batch = Batch(w.starts.data_ptr(), w.lengths.data_ptr(), w.table.data_ptr(), 3, w.table.shape[1], w.table.stride(0))
        tok = lambda t: ctypes.byref(Tokens(t.data_ptr(), t.stride(0), t.stride(1)))
        st = L.nvfp4_cache_attention(tok(q), w.T, Hq, ctypes.byref(cache), ctypes.byref(batch), dim ** -0.5, 1, 0, 0, tok(o),
                                     None, ws.data_ptr() + 256, n, None, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(o, want)
        assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + n:] == 0xA5).all())


def test_a_wait_that_runs_out_is_reported():
    """A build whose keys never come: the kernel for many rows gives up after about a second, says so, frees what it
    holds and leaves the context usable."""
    import ctypes
    from nvfp4_bit_block_gb300.build import build_attention_selftest
    L = ctypes.CDLL(build_attention_selftest())
    w = Work([300], [200], 1, 64, 16, seed=94)
    w.fill()
    q, st = rand((200, 2, 64), BF, 95), ints([0])
    o, p, c = torch.zeros_like(q), ctypes.c_void_p, w.cache
    args = [p(t.data_ptr()) for t in (q, o, c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.alpha, w.starts, w.lengths, w.table)]
    torch.cuda.synchronize()
    assert L.nvfp4_selftest_attend_many(*args, 200, 1, 2, 64, 16, w.table.shape[1], p(st.data_ptr())) == 0
    torch.cuda.synchronize()
    assert st.item() == -8
    r = nv.nvfp4_cache_attention(q, c, *w.batch, want_lse=True)
    check_attention(w, q, r)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("M", [1, 16, 300])
def test_a_linear_layer_right_behind(M, dim):
    """A call whose kernel takes tensor memory before it waits for the attention's: 20 of them, back to back."""
    w = Work([900, 700, 1100], [900, 513, 700], 2, dim, 16, seed=104)
    w.fill()
    q = rand((w.T, 8, dim), BF, 105)
    want = nv.nvfp4_cache_attention(q, w.cache, *w.batch).o
    flags = nv.ROWWISE | nv.SF_SWIZZLED
    operands = []
    for m, seed in ((M, 106), (256, 107)):
        x = rand((m, 256), BF, seed)
        z = nv.nvfp4_quantize(x, nv.nvfp4_amax(x, flags), flags)
        operands += [z.q_row, z.s_row, z.alpha[0:1]]
    lin = lambda: nv.nvfp4_linear(*operands).d
    d = lin().clone()
    for _ in range(20):
        o, e = nv.nvfp4_cache_attention(q, w.cache, *w.batch).o, lin()
    assert torch.equal(o, want) and torch.equal(e, d)


@both_kernels
@pytest.mark.parametrize("news", [[1, 1, 1, 1], [20, 1, 300, 2]])
def test_attention_on_two_streams_at_once(news):
    """Calls that run at the same time have workspaces of their own."""
    w = Work([800, 300, 500, 64], news, 2, 128, 32, seed=96)
    w.fill()
    qs = [rand((w.T, 10, 128), BF, 97 + i) for i in range(4)]
    want = [nv.nvfp4_cache_attention(q, w.cache, *w.batch).o for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [None] * 4
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = nv.nvfp4_cache_attention(qs[i], w.cache, *w.batch).o
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_captured_graphs_share_the_cache():
    """Write and attention captured together, replayed with other tokens and lengths; two graphs in turn."""
    w = Work([64, 40], [1, 1], 1, 64, 16, seed=98)
    w.fill()
    k, v, q = rand((2, 1, 64), BF, 99), rand((2, 1, 64), BF, 100), rand((2, 3, 64), BF, 101)
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.nvfp4_cache_write(k, v, w.cache, *w.batch)
            o = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True)
        graphs.append((g, o))
    for step in range(6):
        w.lengths.copy_(ints([50 + step, 30 + step]))
        for t, s in ((k, 200), (v, 300), (q, 400)):
            t.copy_(rand(t.shape, BF, s + step))
        g, o = graphs[step % 2]
        g.replay()
        w.lens, w.news = [50 + step, 30 + step], [1, 1]
        check_attention(w, q, o)


def test_long_contexts_and_many_sequences():
    """A sequence of 100000 keys among short ones, and 3000 sequences."""
    w = Work([100000, 5, 40000], [1, 1, 2], 1, 64, 64, seed=102)
    w.fill()
    attend(w, 4)
    w = Work([(i * 37) % 90 for i in range(3000)], [1 if i % 7 else 0 for i in range(3000)], 1, 32, 16, seed=103)
    w.lens = [max(n, m) for n, m in zip(w.lens, w.news)]
    w = Work(w.lens, w.news, 1, 32, 16, seed=103)
    w.fill()
    attend(w, 2)


def test_offsets_beyond_32_bits():
    """Pages that lie more than 2^32 bytes from the first."""
    P = 70000
    kc = torch.zeros((P, 1, 512, 128), dtype=torch.uint8, device="cuda")  # 4.6 GB
    vc = kc  # the same bytes serve as values
    sc = torch.full((P, 1, 512, 16), 0x38, dtype=torch.uint8, device="cuda")
    cache = nv.KVCache(kc, sc, vc, sc, torch.ones(2, dtype=F32, device="cuda"))
    far = [69999, 67001, 65537]
    for i, p in enumerate(far):
        kc[p] = torch.randint(0, 256, kc[p].shape, generator=gen(104 + i), device="cuda", dtype=torch.uint8)
    near = nv.KVCache(*(t[far].contiguous() for t in (kc, sc, kc, sc)), cache.alpha)
    for m in (1, 70):
        batch = (ints([0, m]), ints([1300]))
        q = rand((m, 2, 256), BF, 108, 0.1)
        a = nv.nvfp4_cache_attention(q, cache, *batch, ints([far]))
        b = nv.nvfp4_cache_attention(q, near, *batch, ints([[0, 1, 2]]))
        assert torch.equal(a.o, b.o)
        x = nv.nvfp4_cache_read(cache, *batch, ints([far]), tokens=m)
        y = nv.nvfp4_cache_read(near, *batch, ints([[0, 1, 2]]), tokens=m)
        assert torch.equal(x.k, y.k)
