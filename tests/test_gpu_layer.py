"""The operators around the linear layer on the GPU, against their formulas in 64 bits.

Tolerances.  Write u = 2^-24 for the rounding of an fp32 operation and u_out for
that of the result (half the type's spacing: 2^-8 for bf16, u for fp32).  A sum over n values whose
longest chain of additions is c is off by at most c * u * sum|.|; the kernels'
chains are a thread's own values (some tens, at most 2^7 with the tree that
joins the threads at the sizes used here), so sums, means and the few roundings
around them are held to T = 2^-17 = 2^7 u of the sum of magnitudes.  Each test
carries that through the formula: the bound of an element is u_out * |result|
plus T times the magnitudes that entered it.  Activations: the exponential's
argument t is rounded to u|t| and the fast exponential adds 2 units and u|t|
more, which moves p = sigmoid(t) by p (1 - p)(3 u |t|) <= 2 u; with the
products around it act and act' are within 2^-19 (|z| + 1).  The FP4 product is
held to 2^-16 of sum |a b|, the bar of the GEMM's tests.
"""
import math

import numpy as np
import pytest
import torch

import nvfp4_bit_block_gb300 as nv
import synthetic

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
T = 2.0 ** -17
TACT = 2.0 ** -19
TGEMM = 2.0 ** -16
U_OUT = {t: torch.finfo(t).eps / 2 for t in (BF, F32)}
TYPES = [(BF, BF), (F32, BF), (F32, F32), (BF, F32)]


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    nv.build()


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


CANARY = 12345.0


def strided(t, pad, offset):
    """t's values in a wider buffer of canaries: row stride N + pad, first element `offset` elements in."""
    M, N = t.shape
    base = torch.full((offset + M * (N + pad) + 8,), CANARY, dtype=t.dtype, device="cuda")
    v = base[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    v.copy_(t)
    return base, v


def untouched(base, M, N, pad, offset):
    """Every element of the buffer outside the M x N view still holds the canary."""
    want = torch.tensor(CANARY, dtype=base.dtype, device="cuda")
    body = base[offset:offset + M * (N + pad)].view(M, N + pad)
    return bool((base[:offset] == want).all() and (base[offset + M * (N + pad):] == want).all()
                and (body[:, N:] == want).all())


def within(got, ref, tol, what):
    got, tol = got.double(), torch.as_tensor(tol, dtype=torch.float64, device=got.device)
    bad = ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        t = tol.expand_as(ref)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: got "
                             f"{got[i].item()!r}, {ref[i].item()!r} within {t.item():.3g}")


# ---------------------------------------------------------------- layer norm


def norm64(x, gamma, beta, eps):
    x = x.double()
    N = x.shape[1]
    mean = x.sum(1, keepdim=True) / N
    var = ((x - mean) ** 2).sum(1, keepdim=True) / N
    rstd = (var + eps) ** -0.5
    g = gamma.double() if gamma is not None else torch.ones(N, dtype=torch.float64, device=x.device)
    b = beta.double() if beta is not None else torch.zeros(N, dtype=torch.float64, device=x.device)
    return (x - mean) * rstd * g + b, mean, rstd, var, g, b


def check_norm(x, gamma, beta, eps, r, out_dtype):
    y, mean, rstd, var, g, b = norm64(x, gamma, beta, eps)
    off = T * x.double().abs().mean(1, keepdim=True)  # of the mean, hence of x - mean
    rel = T + 0.5 * off ** 2 / (var + eps)            # of rstd
    within(r.mean[:, None], mean, off, "mean")
    within(r.rstd[:, None], rstd, rel * rstd, "rstd")
    within(r.y, y, U_OUT[out_dtype] * y.abs() + (1 + rel) * off * rstd * g.abs() + (rel + T) * ((y - b).abs())
           + T * b.abs(), "y")


SHAPES = [(1, 1), (3, 7), (2, 33), (5, 257), (1, 5120), (7, 1000), (33, 1023), (130, 64), (4, 2731), (3, 8192),
          (2, 20480), (2, 33001), (700, 48), (1, 40000)]


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("M,N", SHAPES)
def test_layernorm(M, N, xt, yt):
    x = rand((M, N), xt, M * 7 + N, 2.0, 0.5)
    gamma, beta = rand((N,), F32, 1, 0.1, 1.0), rand((N,), F32, 2, 0.1)
    r = nv.nvfp4_layernorm(x, gamma, beta, 1e-5, out_dtype=yt)
    assert r.y.dtype is yt and r.amax is None
    check_norm(x, gamma, beta, 1e-5, r, yt)


# enough rows that each block walks over several: every kernel and width, rows of 16-byte pieces and others
MANY_ROWS = [(5003, 64), (3001, 256), (2500, 520), (2001, 1024), (1301, 5120), (1250, 8192), (701, 20480), (650, 32768),
             (620, 33008), (3001, 257), (3000, 1001), (1500, 2731), (1301, 5001), (900, 8191), (650, 12289)]


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("M,N", MANY_ROWS)
def test_layernorm_many_rows(M, N, xt, yt):
    x = rand((M, N), xt, M + 3 * N, 2.0, 0.5)
    gamma, beta = rand((N,), F32, 1, 0.1, 1.0), rand((N,), F32, 2, 0.1)
    r = nv.nvfp4_layernorm(x, gamma, beta, 1e-5, out_dtype=yt, want_amax=True)
    check_norm(x, gamma, beta, 1e-5, r, yt)
    assert r.amax.tolist() == [float(r.y.float().abs().max())] * 2


# rows of each shift against 16-byte boundaries: strides N + pad that are 0, 1, 2, 3 and 4 mod 8, more rows than fit one
# block; N around a chunk's and a block's width
ODD_ROWS = [(259, 7, 0), (300, 48, 1), (1030, 1001, 0), (1217, 1001, 7), (777, 84, 0), (2049, 130, 4), (641, 2731, 4),
            (1300, 1022, 0), (1219, 1025, 1), (601, 4099, 0), (1250, 5113, 0), (1240, 5119, 4), (700, 8193, 0),
            (1001, 2, 0), (999, 3, 0), (1003, 8, 1), (1300, 9, 0)]


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("M,N,pad", ODD_ROWS + [(1301, 8199, 0), (650, 12379, 0), (700, 20479, 1)])
def test_layernorm_odd_rows(M, N, pad, xt, yt):
    """Nothing beside the rows is written, and neighbouring rows' NaN reaches no other."""
    x = rand((M, N), xt, M + 3 * N, 2.0, 0.5)
    gamma, beta = rand((N,), F32, 1, 0.1, 1.0), rand((N,), F32, 2, 0.1)
    xv = strided(x, pad, 0)[1]
    base, out = strided(torch.zeros((M, N), dtype=yt, device="cuda"), pad, 0)
    r = nv.nvfp4_layernorm(xv, gamma, beta, 1e-5, out=out, want_amax=True)
    check_norm(x, gamma, beta, 1e-5, r, yt)
    assert untouched(base, M, N, pad, 0)
    assert r.amax.tolist() == [float(r.y.float().abs().max())] * 2
    clean = r.y.clone()
    xv[M // 2] = float("nan")
    got = nv.nvfp4_layernorm(xv, gamma, beta, 1e-5, out=xv if xt == yt else out).y  # in place
    rows = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[rows], clean[rows])


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (0, 1), (4, 2)])
@pytest.mark.parametrize("xt,yt", TYPES)
def test_layernorm_strides_and_alignment(xt, yt, pad, offset):
    """Rows that start anywhere: nothing outside the view is written."""
    for M, N in ((5, 1000), (3, 257), (9, 5120)):
        x = rand((M, N), xt, 3)
        _, xv = strided(x, pad, offset)
        base, yv = strided(torch.zeros((M, N), dtype=yt, device="cuda"), pad, offset)
        r = nv.nvfp4_layernorm(xv, None, None, 1e-6, out=yv)
        assert r.y is yv
        check_norm(x, None, None, 1e-6, r, yt)
        assert untouched(base, M, N, pad, offset)


@pytest.mark.parametrize("wt", [BF, F32])
def test_layernorm_optional_weights_and_outputs(wt):
    x = rand((6, 520), BF, 4)
    gamma, beta = rand((520,), wt, 5, 0.2, 1.0), rand((520,), wt, 6)
    for g, b in ((gamma, beta), (gamma, None), (None, beta), (None, None)):
        check_norm(x, g, b, 1e-5, nv.nvfp4_layernorm(x, g, b, 1e-5), BF)
    r = nv.nvfp4_layernorm(x, gamma, beta, want_stats=False)
    assert r.mean is None and r.rstd is None
    assert torch.equal(r.y, nv.nvfp4_layernorm(x, gamma, beta).y)


def test_layernorm_in_place():
    for N in (96, 1001, 5120, 40000):
        x = rand((5, N), BF, 7)
        want = nv.nvfp4_layernorm(x, None, None).y
        got = x.clone()
        nv.nvfp4_layernorm(got, None, None, out=got)
        assert torch.equal(got, want), N


def test_layernorm_of_rows_without_spread_and_far_from_zero():
    """Constant rows, a mean a thousand times the spread, and rows of zeros."""
    x = rand((6, 777), F32, 8)
    x[0] = 0.0
    x[1] = 3.0
    x[2] = x[2] + 1000.0
    x[3] = x[3] * 1e-6
    x[4] = -1e4
    x[5] = x[5] * 1e15
    check_norm(x, None, None, 1e-5, nv.nvfp4_layernorm(x, None, None, 1e-5), F32)
    r = nv.nvfp4_layernorm(x[:2].contiguous(), None, None, 1e-5)
    assert bool((r.y[0] == 0).all())
    one = nv.nvfp4_layernorm(rand((4, 1), F32, 9, 5.0), None, None, 1e-5)  # a single column is its own mean
    assert bool((one.y == 0).all())


@pytest.mark.parametrize("N", [64, 1023, 5120, 33000])
def test_layernorm_nan_and_inf_stay_in_their_rows(N):
    x = rand((8, N), BF, 10)
    clean = nv.nvfp4_layernorm(x).y
    y = x.clone()
    y[2, N // 2] = float("nan")
    y[5, N - 1] = float("inf")
    got = nv.nvfp4_layernorm(y, want_amax=True)
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(got.y[keep], clean[keep])
    assert bool(got.y[2].isnan().all())
    assert bool(got.y[5].isnan().all() or not got.y[5].isfinite().all())
    assert bool(got.amax.isnan().all())


@pytest.mark.parametrize("M,N", [(1, 64), (1, 5120), (3, 1008), (17, 5120), (1000, 512), (40, 33008)])
def test_layernorm_amax_is_the_quantizers(M, N):
    x = rand((M, N), BF, 11, 3.0)
    r = nv.nvfp4_layernorm(x, rand((N,), F32, 12, 0.3, 1.0), None, want_amax=True)
    assert torch.equal(r.amax, nv.nvfp4_amax(r.y, nv.ROWWISE))
    q = nv.nvfp4_quantize(r.y, r.amax, nv.ROWWISE)
    assert int(q.status.item()) == 0


def test_layernorm_empty():
    r = nv.nvfp4_layernorm(torch.empty((0, 64), dtype=BF, device="cuda"), want_amax=True)
    assert r.y.shape == (0, 64) and r.amax.tolist() == [0.0, 0.0]
    r = nv.nvfp4_layernorm(torch.empty((3, 0), dtype=BF, device="cuda"), want_amax=True)
    assert r.y.shape == (3, 0) and r.amax.tolist() == [0.0, 0.0]


# ---------------------------------------------------------------- its gradient


def norm_grad64(dy, x, mean, rstd, gamma, dres):
    dy, x = dy.double(), x.double()
    N = x.shape[1]
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy * gamma.double() if gamma is not None else dy
    dx = rstd.double()[:, None] * (g - g.sum(1, keepdim=True) / N - xh * (g * xh).sum(1, keepdim=True) / N)
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0), g, xh


def check_norm_grad(dy, x, mean, rstd, gamma, dres, r):
    dx, dg, db, g, xh = norm_grad64(dy, x, mean, rstd, gamma, dres)
    mag = g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    tol = U_OUT[x.dtype] * dx.abs() + T * rstd.double()[:, None] * mag
    if dres is not None:
        tol = tol + T * dres.double().abs()
    within(r.dx, dx, tol, "dx")
    if r.dgamma is not None:
        within(r.dgamma, dg, T * (dy.double() * xh).abs().sum(0), "dgamma")
    if r.dbeta is not None:
        within(r.dbeta, db, T * dy.double().abs().sum(0), "dbeta")


def stats(x, eps=1e-5):
    _, mean, rstd, *_ = norm64(x, None, None, eps)
    return mean[:, 0].float(), rstd[:, 0].float()


@pytest.mark.parametrize("xt,dt", TYPES)
@pytest.mark.parametrize("M,N", SHAPES + [(1000, 520), (317, 5120)])
def test_layernorm_backward(M, N, xt, dt):
    x, dy = rand((M, N), xt, M + N, 2.0, 0.3), rand((M, N), dt, M + N + 1, 1e-3)
    gamma = rand((N,), F32, 13, 0.2, 1.0)
    dres = rand((M, N), xt, 14, 1e-3) if (M + N) % 2 else None
    mean, rstd = stats(x)
    check_norm_grad(dy, x, mean, rstd, gamma, dres, nv.nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, dres))


@pytest.mark.parametrize("xt,dt", TYPES)
@pytest.mark.parametrize("M,N", MANY_ROWS + [(1217, 3000), (1300, 4104), (1303, 10240)])
def test_layernorm_backward_many_rows(M, N, xt, dt):
    x, dy = rand((M, N), xt, M + N, 2.0, 0.3), rand((M, N), dt, M + N + 1, 1e-3)
    gamma = rand((N,), F32, 13, 0.2, 1.0)
    mean, rstd = stats(x)
    for dres in (None, rand((M, N), xt, 14, 1e-3)):
        check_norm_grad(dy, x, mean, rstd, gamma, dres, nv.nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, dres))


@pytest.mark.parametrize("M,N", [(1301, 5120), (1300, 1001), (640, 20480)])
def test_layernorm_backward_in_place_many_rows(M, N):
    x, dy, dres = rand((M, N), BF, 21), rand((M, N), BF, 22), rand((M, N), BF, 23)
    mean, rstd = stats(x)
    want = nv.nvfp4_layernorm_backward(dy, x, mean, rstd, None, dres)
    for k in (0, 1):
        d, e = dy.clone(), dres.clone()
        got = nv.nvfp4_layernorm_backward(d, x, mean, rstd, None, e, out=(d, e)[k])
        assert torch.equal(got.dx, want.dx) and torch.equal(got.dgamma, want.dgamma)
        assert torch.equal(got.dbeta, want.dbeta)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (0, 1)])
@pytest.mark.parametrize("xt,dt", TYPES)
def test_layernorm_backward_strides_and_alignment(xt, dt, pad, offset):
    for M, N in ((5, 1000), (37, 257), (9, 5120)):
        x, dy, dres = rand((M, N), xt, 15), rand((M, N), dt, 16), rand((M, N), xt, 17)
        mean, rstd = stats(x)
        base, out = strided(torch.zeros_like(x), pad, offset)
        r = nv.nvfp4_layernorm_backward(strided(dy, pad, offset)[1], strided(x, pad, offset)[1], mean, rstd, None,
                                        strided(dres, pad, offset)[1], out=out)
        check_norm_grad(dy, x, mean, rstd, None, dres, r)
        assert untouched(base, M, N, pad, offset)


@pytest.mark.parametrize("xt,dt", TYPES)
@pytest.mark.parametrize("M,N,pad", ODD_ROWS)
def test_layernorm_backward_odd_rows(M, N, pad, xt, dt):
    """Nothing beside the rows is written, and neighbouring rows' NaN reaches no other."""
    x, dy, dres = rand((M, N), xt, M + N, 2.0, 0.3), rand((M, N), dt, M + N + 1, 1e-3), rand((M, N), xt, 14, 1e-3)
    gamma = rand((N,), F32, 13, 0.2, 1.0)
    mean, rstd = stats(x)
    base, out = strided(torch.zeros_like(x), pad, 0)
    xv, dyv, resv = strided(x, pad, 0)[1], strided(dy, pad, 0)[1], strided(dres, pad, 0)[1]
    check_norm_grad(dy, x, mean, rstd, gamma, None, nv.nvfp4_layernorm_backward(dyv, xv, mean, rstd, gamma, out=out))
    r = nv.nvfp4_layernorm_backward(dyv, xv, mean, rstd, gamma, resv, out=out)
    check_norm_grad(dy, x, mean, rstd, gamma, dres, r)
    assert untouched(base, M, N, pad, 0)
    clean = r.dx.clone()
    xv[M // 2] = float("nan")
    dyv[M // 3] = float("inf")
    got = nv.nvfp4_layernorm_backward(dyv, xv, mean, rstd, gamma, resv, out=resv).dx  # in place
    rows = torch.arange(M, device="cuda")
    rows = (rows != M // 2) & (rows != M // 3)
    assert torch.equal(got[rows], clean[rows])


def test_layernorm_backward_options():
    x, dy, gamma = rand((50, 640), BF, 18), rand((50, 640), BF, 19), rand((640,), BF, 20, 0.1, 1.0)
    mean, rstd = stats(x)
    full = nv.nvfp4_layernorm_backward(dy, x, mean, rstd, gamma)
    check_norm_grad(dy, x, mean, rstd, gamma, None, full)
    r = nv.nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, want_dgamma=False)
    assert r.dgamma is None and torch.equal(r.dbeta, full.dbeta) and torch.equal(r.dx, full.dx)
    r = nv.nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, want_dbeta=False)
    assert r.dbeta is None and torch.equal(r.dgamma, full.dgamma) and torch.equal(r.dx, full.dx)
    r = nv.nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, want_dgamma=False, want_dbeta=False)
    assert r.dgamma is None and r.dbeta is None and torch.equal(r.dx, full.dx)


@pytest.mark.parametrize("N", [96, 1001, 5120, 40000])
def test_layernorm_backward_in_place(N):
    """dx in dy's or dres's place."""
    x, dy, dres = rand((9, N), BF, 21), rand((9, N), BF, 22), rand((9, N), BF, 23)
    mean, rstd = stats(x)
    want = nv.nvfp4_layernorm_backward(dy, x, mean, rstd, None, dres)
    for k in (0, 1):
        d, e = dy.clone(), dres.clone()
        got = nv.nvfp4_layernorm_backward(d, x, mean, rstd, None, e, out=(d, e)[k])
        assert torch.equal(got.dx, want.dx) and torch.equal(got.dgamma, want.dgamma)
        assert torch.equal(got.dbeta, want.dbeta)


def test_layernorm_backward_empty():
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    s = torch.empty(0, device="cuda")
    r = nv.nvfp4_layernorm_backward(e, e, s, s)
    assert r.dx.shape == (0, 64) and bool((r.dgamma == 0).all()) and bool((r.dbeta == 0).all())


def test_layernorm_gradient_against_differences():
    """L = sum(w * y): the kernel's gradient along a direction against central
    differences of the kernel's forward pass.  With step h the differences are
    off by the forward's rounding, about sqrt(n) * 2^-22 * |w y| / h, and by the
    third derivative, O(h^2); both are below 1 % of the slope along the
    gradient itself at h = 2^-7."""
    M, N, h = 16, 257, 2.0 ** -7
    x, w = rand((M, N), F32, 24), rand((M, N), F32, 25)
    gamma, beta = rand((N,), F32, 26, 0.2, 1.0), rand((N,), F32, 27)
    f = nv.nvfp4_layernorm(x, gamma, beta)
    r = nv.nvfp4_layernorm_backward(w, x, f.mean, f.rstd, gamma)

    def loss(x, gamma, beta):
        return float((w.double() * nv.nvfp4_layernorm(x, gamma, beta).y.double()).sum())
    for at, grad in ((0, r.dx), (1, r.dgamma), (2, r.dbeta)):
        v = grad / grad.square().mean().sqrt()
        args = [[x, gamma, beta] for _ in (0, 1)]
        args[0][at], args[1][at] = args[0][at] + h * v, args[1][at] - h * v
        slope = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        want = float((grad.double() * v.double()).sum())
        assert abs(slope - want) <= 0.01 * abs(want), (at, slope, want)


# ---------------------------------------------------------------- activation


def act64(z, act):
    if act == nv.ACT_RELU:
        return z.clamp(min=0)
    if act == nv.ACT_GELU:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == nv.ACT_GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == nv.ACT_SILU:
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    """Derivative by automatic differentiation of the 64-bit formula (relu: 0 at 0)."""
    if act == nv.ACT_RELU:
        return (z > 0).double()
    if act == nv.ACT_NONE:
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    act64(z, act).sum().backward()
    return z.grad


def check_act_grad(dy, z, act, r):
    d = dy.double()
    s = slope64(z.double(), act)
    zz = z.double().abs().clamp(max=16)  # beyond that the slope is 0 or 1 to fp32
    if r.dz is not None:
        within(r.dz, d * s, U_OUT[dy.dtype] * (d * s).abs() + TACT * (1 + zz) * d.abs(), "dz")
    if r.dbias is not None:
        within(r.dbias, (d * s).sum(0), (TACT * (1 + zz) * d.abs()).sum(0) + T * (d * s).abs().sum(0), "dbias")


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("dt", [BF, F32])
def test_act_backward(act, dt):
    for M, N in ((1, 1), (3, 7), (67, 1001), (1, 20480), (300, 33), (129, 1024), (1000, 264), (2, 33001), (517, 2056),
                 (5000, 72), (4001, 2048), (3000, 1001)):
        dy, z = rand((M, N), dt, M + N, 1e-3), rand((M, N), dt, N, 2.0)
        check_act_grad(dy, z, act, nv.nvfp4_act_backward(dy, z, act))


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (0, 1)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_act_backward_strides_and_alignment(dt, pad, offset):
    for M, N in ((37, 257), (9, 5120), (260, 72)):
        dy, z = rand((M, N), dt, 30), rand((M, N), dt, 31)
        base, out = strided(torch.zeros_like(dy), pad, offset)
        r = nv.nvfp4_act_backward(strided(dy, pad, offset)[1], strided(z, pad, offset)[1], nv.ACT_GELU, out=out)
        check_act_grad(dy, z, nv.ACT_GELU, r)
        assert untouched(base, M, N, pad, offset)


@pytest.mark.parametrize("act", [nv.ACT_NONE, nv.ACT_RELU, nv.ACT_GELU_TANH])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,N,pad", ODD_ROWS)
def test_act_backward_odd_rows(M, N, pad, dt, act):
    """Nothing beside the rows is written, and neighbouring rows' NaN reaches no other."""
    dy, z = rand((M, N), dt, M + N, 1e-3), rand((M, N), dt, N, 2.0)
    base, out = strided(torch.zeros_like(dy), pad, 0)
    dyv, zv = strided(dy, pad, 0)[1], strided(z, pad, 0)[1]
    r = nv.nvfp4_act_backward(dyv, zv, act, out=out)
    check_act_grad(dy, z, act, r)
    assert untouched(base, M, N, pad, 0)
    clean = r.dz.clone()
    dyv[M // 2] = float("nan")
    got = nv.nvfp4_act_backward(dyv, zv, act, out=dyv).dz  # in place
    rows = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[rows], clean[rows])


def test_act_backward_options_and_in_place():
    dy, z = rand((70, 1000), BF, 32), rand((70, 1000), BF, 33)
    full = nv.nvfp4_act_backward(dy, z, nv.ACT_SILU)
    r = nv.nvfp4_act_backward(dy, z, nv.ACT_SILU, want_dbias=False)
    assert r.dbias is None and torch.equal(r.dz, full.dz)
    r = nv.nvfp4_act_backward(dy, z, nv.ACT_SILU, want_dz=False)
    assert r.dz is None and torch.equal(r.dbias, full.dbias)
    for k in (0, 1):
        a, b = dy.clone(), z.clone()
        r = nv.nvfp4_act_backward(a, b, nv.ACT_SILU, out=(a, b)[k])
        assert torch.equal(r.dz, full.dz) and torch.equal(r.dbias, full.dbias)
    r = nv.nvfp4_act_backward(dy, None, nv.ACT_NONE, want_dz=False)  # a bias gradient alone
    check_act_grad(dy, z, nv.ACT_NONE, r)
    assert torch.equal(nv.nvfp4_act_backward(dy, None, nv.ACT_NONE).dz, dy)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_act_backward(dy, None, nv.ACT_GELU)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_act_backward(dy, z, 7)
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    assert bool((nv.nvfp4_act_backward(e, e, nv.ACT_GELU).dbias == 0).all())


@pytest.mark.parametrize("act", range(1, 5))
def test_act_backward_extremes(act):
    """Large, infinite and tiny z have the limits of the derivative; NaN stays NaN."""
    z = torch.tensor([[0.0, -0.0, 1e-30, 1e30, -1e30, 1e4, -1e4, 30.0, -30.0, float("inf"), float("-inf"),
                       float("nan")]], device="cuda")
    r = nv.nvfp4_act_backward(torch.ones_like(z), z, act).dz[0]
    half = 0.0 if act == nv.ACT_RELU else 0.5
    tiny = 1.0 if act == nv.ACT_RELU else 0.5
    want = torch.tensor([half, half, tiny, 1, 0, 1, 0, 1, 0, 1, 0], device="cuda")
    assert bool(((r[:-1] - want).abs() <= 2.0 ** -19).all()), r
    assert bool(r[-1].isnan())


# ---------------------------------------------------------------- linear


def values(q, sf, K):
    """Codes times block scales in 64 bits, from the plain layouts' definition."""
    R = q.shape[0]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device=q.device)
    v = grid[torch.stack([q & 15, q >> 4], 2).long()].view(R, K // 16, 16)
    r = torch.arange(R, device=q.device)[:, None]
    c = torch.arange(K // 16, device=q.device)[None, :]
    at = ((r // 128) * (sf.shape[1] // 4) + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4
    return (v * sf.reshape(-1)[at].view(torch.float8_e4m3fn).double()[:, :, None]).view(R, K)


def operand(R, K, seed, scale=1.0, garbage=True):
    """A quantized R x K tensor; the scale layout's padding holds E4M3 NaNs (any bytes may be there)."""
    bits = synthetic.activation_outlier_channels(R, K, seed, frac=0.01)
    x = torch.from_numpy(bits.view(np.int16)).view(BF).cuda() * scale
    flags = nv.ROWWISE | nv.SF_SWIZZLED
    q = nv.nvfp4_quantize(x, nv.nvfp4_amax(x, flags), flags)
    assert int(q.status.item()) == 0
    if garbage:
        r = torch.arange(R, device="cuda")[:, None]
        c = torch.arange(K // 16, device="cuda")[None, :]
        C4 = q.s_row.shape[1] // 4
        pad = torch.ones(q.s_row.numel(), dtype=torch.bool, device="cuda")
        pad[(((r // 128) * C4 + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4).reshape(-1)] = False
        q.s_row.view(-1)[pad] = 0x7F
    return q.q_row, q.s_row, q.alpha[0:1]


def check_linear(a, b, K, r, bias=None, act=0, residual=None, dtype=BF):
    xa, xb = values(a[0], a[1], K), values(b[0], b[1], K)
    scale = a[2].double() * b[2].double()
    z = xa @ xb.t() * scale
    tz = TGEMM * (xa.abs() @ xb.abs().t()) * scale.abs()
    if bias is not None:
        z = z + bias.double()
        tz = tz + 4 * U * (z.abs() + bias.double().abs())
    d = act64(z, act)
    td = 1.2 * tz + (TACT * (1 + z.abs()) if act else 0)
    if residual is not None:
        d = d + residual.double()
        td = td + 2 * U * residual.double().abs()
    within(r.d, d, td + U_OUT[dtype] * d.abs(), "d")
    if r.z is not None:
        within(r.z, z, tz + U_OUT[dtype] * z.abs(), "z")


LINEAR = [(1, 1, 32), (1, 40, 64), (1, 5120, 1024), (3, 130, 96), (8, 256, 256), (16, 200, 2080), (17, 1000, 1056),
          (24, 513, 4096), (33, 128, 544), (64, 640, 512), (65, 257, 288), (127, 384, 320), (128, 128, 256),
          (129, 1111, 992), (200, 96, 7200), (256, 512, 1024), (333, 1000, 1056), (300, 2600, 1536),
          (2048, 1280, 768), (1000, 31, 64),
          # whole output tiles over the GPU, with every edge: tokens, features, K % 64, a second band that is not there
          (1000, 2600, 544), (2050, 2177, 96), (4000, 1000, 1312), (1500, 1921, 32)]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(M, N, K):
    a, b = operand(M, K, M + K), operand(N, K, N + K + 1, 0.05)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bias = rand((N,), F32, 40, 0.3)
    r = nv.nvfp4_linear(*a, *b, bias=bias, act=nv.ACT_GELU_TANH, want_z=True, want_amax=True, status=status)
    assert r.d.dtype is BF and int(status.item()) == 0
    check_linear(a, b, K, r, bias, nv.ACT_GELU_TANH)
    assert r.amax.tolist() == [float(r.d.float().abs().max())] * 2
    res = rand((M, N), F32, 41)
    r = nv.nvfp4_linear(*a, *b, residual=res, out_dtype=F32, status=status)
    assert r.z is None and r.amax is None and int(status.item()) == 0
    check_linear(a, b, K, r, residual=res, dtype=F32)


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (20, 300, 512), (140, 300, 512), (1300, 2056, 96)])
@pytest.mark.parametrize("act", range(5))
def test_linear_every_epilogue(M, N, K, act):
    a, b = operand(M, K, 50), operand(N, K, 51, 0.05)
    for dt in (BF, F32):
        for bias in (None, rand((N,), F32, 52), rand((N,), BF, 53)):
            for res in (None, rand((M, N), dt, 54)):
                r = nv.nvfp4_linear(*a, *b, bias=bias, act=act, residual=res, out_dtype=dt, want_z=True)
                check_linear(a, b, K, r, bias, act, res, dt)


@pytest.mark.parametrize("M,N,K", [(2050, 5001, 96), (2050, 5000, 544), (300, 20001, 1056), (2560, 5120, 64)])
def test_linear_several_tiles_per_pair(M, N, K):
    """More tiles than pairs of SMs, outputs with and without rows of whole vectors, everything on."""
    a, b = operand(M, K, M + K), operand(N, K, N + K)
    bias = rand((N,), F32, 3)
    for dt in (BF, F32):
        res = rand((M, N), dt, 5)
        for r, z in ((None, True), (res, False), (res, True)):
            got = nv.nvfp4_linear(*a, *b, bias=bias, act=nv.ACT_SILU, residual=r, out_dtype=dt, want_z=z,
                                  want_amax=dt is BF)
            check_linear(a, b, K, got, bias, nv.ACT_SILU, r, dt)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (0, 1), (2, 0)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_strides_and_alignment(dt, pad, offset):
    for M, N, K in ((2, 200, 128), (40, 257, 160), (150, 264, 512), (1100, 2600, 96)):
        a, b, res = operand(M, K, 60), operand(N, K, 61), rand((M, N), dt, 62)
        base, out = strided(torch.zeros((M, N), dtype=dt, device="cuda"), pad, offset)
        r = nv.nvfp4_linear(*a, *b, residual=strided(res, pad, offset)[1], out=out)
        check_linear(a, b, K, r, residual=res, dtype=dt)
        assert untouched(base, M, N, pad, offset)
        base, out = strided(res, pad, offset)  # the residual stream updated in place
        assert torch.equal(nv.nvfp4_linear(*a, *b, residual=out, out=out).d, r.d)
        assert untouched(base, M, N, pad, offset)


def test_linear_equals_the_gemm():
    """Without an epilogue: the same numbers as nvfp4_gemm, at sizes that it takes."""
    for M, N, K in ((128, 256, 512), (384, 1280, 2048)):
        a, b = operand(M, K, 70), operand(N, K, 71)
        want = nv.nvfp4_gemm(*a, *b)
        got = nv.nvfp4_linear(*a, *b, out_dtype=F32).d
        xa, xb = values(a[0], a[1], K).abs(), values(b[0], b[1], K).abs()
        within(got, want.double(), 2 * TGEMM * (xa @ xb.t()) * a[2].double() * b[2].double(), "d")


@pytest.mark.parametrize("M,N", [(1, 200), (30, 200), (300, 200), (1100, 2600)])
def test_linear_zero_and_extreme_operands(M, N):
    """All-zero operands give act(bias) + residual; the largest codes and scales do not overflow."""
    K = 320
    a, b = operand(M, K, 80), operand(N, K, 81)
    za = (torch.zeros_like(a[0]), a[1], a[2])
    bias, res = rand((N,), F32, 82), rand((M, N), BF, 83)
    r = nv.nvfp4_linear(*za, *b, bias=bias, act=nv.ACT_RELU, residual=res)
    check_linear(za, b, K, r, bias, nv.ACT_RELU, res)
    top = (torch.full_like(a[0], 0x77), torch.full_like(a[1], 0x7E), torch.ones(1, device="cuda"))
    tob = (torch.full_like(b[0], 0xF7), torch.full_like(b[1], 0x7E), torch.ones(1, device="cuda"))
    check_linear(top, tob, K, nv.nvfp4_linear(*top, *tob, out_dtype=F32), dtype=F32)


def test_linear_nan_scale_stays_in_its_row():
    """An E4M3 NaN scale of one token (or one weight row) makes that row (column) NaN and no other."""
    for M, N in ((4, 300), (200, 300), (1100, 2600)):
        K = 512
        a, b = operand(M, K, 84, garbage=False), operand(N, K, 85, garbage=False)
        clean = nv.nvfp4_linear(*a, *b, out_dtype=F32).d
        sa, sb = a[1].clone(), b[1].clone()
        sa.view(-1)[2 * 16] = 0x7F            # row 2, block 0
        sb.view(-1)[5 * 16 + 512 + 1] = 0x7F  # row 5, block 5
        got = nv.nvfp4_linear(a[0], sa, a[2], b[0], sb, b[2], out_dtype=F32).d
        nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
        nan[2] = True
        nan[:, 5] = True
        assert bool(got[nan].isnan().all()) and torch.equal(got[~nan], clean[~nan])


def test_linear_empty_and_refusals():
    a, b = operand(16, 64, 86), operand(32, 64, 87)
    e = torch.empty((0, 32), dtype=torch.uint8, device="cuda")
    r = nv.nvfp4_linear(e, torch.empty((0, 4), dtype=torch.uint8, device="cuda"), a[2], *b, want_amax=True)
    assert r.d.shape == (0, 32) and r.amax.tolist() == [0.0, 0.0]
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_linear(*a, *b, act=9)
    with pytest.raises(ValueError, match="sfa"):
        nv.nvfp4_linear(a[0], a[1][:, :2], a[2], *b)
    with pytest.raises(TypeError, match="want_amax"):
        nv.nvfp4_linear(*a, *b, out_dtype=F32, want_amax=True)
    with pytest.raises(TypeError):
        nv.nvfp4_linear(*a, *b, residual=rand((16, 32), F32, 1))
    with pytest.raises(ValueError):
        nv.nvfp4_linear(*a, *b, residual=rand((16, 31), BF, 1))
    with pytest.raises(ValueError):
        nv.nvfp4_linear(*a, *b, bias=rand((31,), F32, 1))
    q = torch.zeros((4, 24), dtype=torch.uint8, device="cuda")  # K = 48
    s = torch.zeros((128, 4), dtype=torch.uint8, device="cuda")
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_linear(q, s, a[2], q, s, a[2])


@pytest.mark.parametrize("M,N", [(5, 300), (1100, 2600)])
def test_linear_wait_timeout_is_reported_and_the_context_stays_usable(M, N):
    """Both kernels in a build whose copies are never issued (test-only
    library): every bounded wait runs out, the kernel reports
    NVFP4_ERR_PIPELINE and gives its tensor memory back, and the next call on the
    same context is correct."""
    import ctypes
    from nvfp4_bit_block_gb300.build import build_layer_selftest
    L = ctypes.CDLL(build_layer_selftest())
    p, i64 = ctypes.c_void_p, ctypes.c_int64
    L.nvfp4_test_linear_no_copies.argtypes = [p] * 6 + [i64] * 3 + [p] * 5
    L.nvfp4_test_linear_no_copies_workspace.argtypes = [i64] * 3
    L.nvfp4_test_linear_no_copies_workspace.restype = i64
    K = 2048
    a, b = operand(M, K, 120), operand(N, K, 121)
    ws = torch.empty(max(16, L.nvfp4_test_linear_no_copies_workspace(M, N, K)), dtype=torch.uint8, device="cuda")
    d, res = torch.zeros((M, N), dtype=BF, device="cuda"), rand((M, N), BF, 122)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.nvfp4_test_linear_no_copies(*[t.data_ptr() for t in (*a, *b)], M, N, K, res.data_ptr(), d.data_ptr(),
                                         ws.data_ptr(), status.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert int(status.item()) == -8
    status.zero_()
    r = nv.nvfp4_linear(*a, *b, residual=res, status=status)
    assert int(status.item()) == 0
    check_linear(a, b, K, r, residual=res)


# ---------------------------------------------------------------- all of them


def everything(seed):
    """One call of each operator: a list of tensors."""
    x, dy = rand((300, 1536), BF, seed), rand((300, 1536), BF, seed + 1, 1e-3)
    f = nv.nvfp4_layernorm(x, want_amax=True)
    g = nv.nvfp4_layernorm_backward(dy, x, f.mean, f.rstd)
    out = [f.y, f.mean, f.rstd, f.amax, g.dx, g.dgamma, g.dbeta]
    for M, N in ((1, 640), (40, 640), (300, 640), (1100, 2600)):
        a, b = operand(M, 1536, seed + 2), operand(N, 1536, seed + 3)
        r = nv.nvfp4_linear(*a, *b, act=nv.ACT_GELU, want_z=True, want_amax=True)
        out += [r.d, r.z, r.amax]
    t = nv.nvfp4_act_backward(dy, x, nv.ACT_GELU)
    return out + [t.dz, t.dbias]


def test_the_same_call_gives_the_same_bits():
    first = everything(90)
    for _ in range(3):
        for p, q in zip(first, everything(90)):
            assert torch.equal(p, q)


def test_other_streams():
    """Each call on a stream of its own, while the default stream is busy."""
    want = everything(91)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = rand((300, 1536), BF, 91)
    big = torch.randn(4096, 4096, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        big = big @ big * 1e-3
    f = nv.nvfp4_layernorm(x, want_amax=True, stream=s)
    h = nv.nvfp4_layernorm(x, want_amax=True, stream=s.cuda_stream)
    with torch.cuda.stream(s):
        got = everything(91)
    s.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    assert torch.equal(f.y, want[0]) and torch.equal(h.y, want[0])
    torch.cuda.synchronize()


def test_capture_in_a_graph():
    """The calls can be captured and replayed on new inputs."""
    x, dy = rand((200, 1024), BF, 92), rand((200, 1024), BF, 93)
    a, b = operand(20, 1024, 94), operand(320, 1024, 95)

    def step():
        f = nv.nvfp4_layernorm(x, want_amax=True)
        g = nv.nvfp4_layernorm_backward(dy, x, f.mean, f.rstd)
        r = nv.nvfp4_linear(*a, *b, want_amax=True)
        t = nv.nvfp4_act_backward(dy, x, nv.ACT_SILU)
        return [f.y, f.amax, g.dx, g.dgamma, r.d, r.amax, t.dz, t.dbias]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (96, 97):
        x.copy_(rand((200, 1024), BF, seed))
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(outs, step()):
            assert torch.equal(p, q)


def test_offsets_beyond_32_bits():
    """Rows that lie more than 2^32 bytes (and 2^31 elements) into their buffers."""
    M, N, ld = 33000, 128, 1 << 16
    wide = torch.empty((M, ld), dtype=BF, device="cuda")
    out = torch.empty((M, ld), dtype=BF, device="cuda")
    x, dy = rand((M, N), BF, 98), rand((M, N), BF, 99)
    wide[:, :N], wide[:, 256:256 + N] = x, dy
    xv, dyv, ov = wide[:, :N], wide[:, 256:256 + N], out[:, 512:512 + N]
    want = nv.nvfp4_layernorm(x)
    assert torch.equal(nv.nvfp4_layernorm(xv, out=ov).y, want.y)
    g = nv.nvfp4_layernorm_backward(dy, x, want.mean, want.rstd)
    got = nv.nvfp4_layernorm_backward(dyv, xv, want.mean, want.rstd, out=ov)
    assert torch.equal(got.dx, g.dx) and torch.equal(got.dgamma, g.dgamma)
    t = nv.nvfp4_act_backward(dy, x, nv.ACT_GELU)
    got = nv.nvfp4_act_backward(dyv, xv, nv.ACT_GELU, out=ov)
    assert torch.equal(got.dz, t.dz) and torch.equal(got.dbias, t.dbias)
    a, b = operand(M, 64, 100), operand(N, 64, 101)
    d = nv.nvfp4_linear(*a, *b, residual=x)
    assert torch.equal(nv.nvfp4_linear(*a, *b, residual=xv, out=ov).d, d.d)


# ---------------------------------------------------------------- together


def test_feed_forward_example():
    """All operators with the quantizer in one block, forward, backward and for
    one token, against the same block in fp32.  Rounding to the E2M1 grid costs a
    normal operand about a tenth of its norm, a product of two of them 0.14, and
    the deepest gradient here has three such products behind it: below 0.14 *
    sqrt(3) + the norms' own; a wrong operand, layout or gradient is off by 1."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for name, v in m.run(288, 640, 1536).items():
        assert v <= 0.35, (name, v)
