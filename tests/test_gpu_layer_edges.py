"""The operators around the linear layer where they are easily wrong: host threads,
streams, argument ranges, rows without spread, long sums, the tail of the
Gaussian, scratch memory of exactly the size asked for.  Tolerances as in
test_gpu_layer.py unless a test derives its own."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300 import layer
from test_gpu_layer import (BF, F32, U, act64, check_act_grad, check_linear, check_norm, check_norm_grad, operand, rand,
                            slope64, stats, strided, untouched)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    nv.build()


# ---------------------------------------------------------------- host threads


def test_concurrent_host_threads_with_rows_of_different_widths():
    """C callers launch from several threads at once.  Rows of different widths
    run in the same kernel with different amounts of shared memory; no thread's
    launch may depend on what another has just asked for."""
    L = nv.layer_lib()
    M, rounds, faults = 620, 400, []
    jobs = []
    for N in (1032, 5120, 8192, 5120, 8192):
        x, y = rand((M, N), F32, N), torch.empty((M, N), device="cuda")
        jobs.append((lambda s, x=x, y=y, N=N: L.nvfp4_layernorm(x.data_ptr(), M, N, N, 0, None, None, 0, 1e-5,
                                                                y.data_ptr(), N, 0, None, None, None, s),
                     y, nv.nvfp4_layernorm(x).y))
    for N in (264, 5120, 2048):
        x, dy, dx = rand((M, N), F32, N), rand((M, N), F32, N + 1), torch.empty((M, N), device="cuda")
        mean, rstd = stats(x)
        n = L.nvfp4_layernorm_backward_workspace(M, N)
        ws, sums = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty((2, N), device="cuda")
        jobs.append((lambda s, x=x, dy=dy, dx=dx, mean=mean, rstd=rstd, ws=ws, sums=sums, n=n, N=N:
                     L.nvfp4_layernorm_backward(dy.data_ptr(), N, 0, x.data_ptr(), N, 0, M, N, mean.data_ptr(),
                                                rstd.data_ptr(), None, 0, dy.data_ptr(), N, dx.data_ptr(), N,
                                                sums[0].data_ptr(), sums[1].data_ptr(), ws.data_ptr(), n, s),
                     dx, nv.nvfp4_layernorm_backward(dy, x, mean, rstd, None, dy).dx))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(call):
        s = torch.cuda.Stream()
        start.wait()
        for k in range(rounds):
            status = call(s.cuda_stream)
            if status:
                faults.append((k, status))
                return
        s.synchronize()

    threads = [threading.Thread(target=work, args=(j[0],)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults, faults
    for _, got, want in jobs:
        assert torch.equal(got, want)


# ---------------------------------------------------------------- streams


def test_the_raw_handle_of_the_default_stream():
    """torch.cuda.default_stream().cuda_stream is 0: given as a raw handle it is the
    default stream, behind what was put there before."""
    assert torch.cuda.default_stream().cuda_stream == 0
    new = rand((700, 512), BF, 1)
    want = nv.nvfp4_layernorm(new).y
    x = torch.zeros_like(new)
    big = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    for _ in range(10):  # some 100 ms
        big = big @ big * 1e-3
    x.copy_(new)
    got = nv.nvfp4_layernorm(x, stream=0).y
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # whatever stream is current
        with layer._entered(0, x):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        assert torch.cuda.current_stream() == side


# ---------------------------------------------------------------- arguments


@pytest.mark.parametrize("act", [2 ** 32, 2 ** 32 + 2, -2 ** 32, 2 ** 63, -2 ** 200])
def test_activations_beyond_32_bits_are_refused(act):
    a, b, x = operand(16, 64, 1), operand(32, 64, 2), rand((4, 32), F32, 3)
    for call in (lambda: nv.nvfp4_linear(*a, *b, act=act), lambda: nv.nvfp4_act_backward(x, x, act)):
        with pytest.raises(nv.Nvfp4Error) as e:
            call()
        assert e.value.status == -4


# ---------------------------------------------------------------- rows without spread


def exact_constants(N):
    """Whole numbers below 256 whose sum over N fp32 values is exact in any order, and
    whose sum times the rounded 1 / N is not the number (where there are some)."""
    inv = np.float32(1) / np.float32(N)
    c = [k for k in range(1, 256) if np.float32(N * k) * inv != np.float32(k)]
    return (c or [3])[:5] + [255]


# every kernel: few rows and many, vectors, single values and rows by classes, up to the longest
CONSTANT = [(5, 56), (5, 408), (5, 1128), (5, 9024), (5, 17704), (700, 56), (700, 408), (700, 1128), (700, 9024),
            (700, 20504), (5, 307), (5, 647), (5, 2213), (5, 3081), (5, 6145), (5, 12289), (700, 1543), (700, 3081),
            (5, 34263)]


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("M,N", CONSTANT)
def test_layernorm_of_constant_rows_is_beta(M, N, xt):
    """A row of one value far from zero has that mean and no spread: where its sum is
    exact, so are the mean and y = beta."""
    c = torch.tensor(exact_constants(N), device="cuda", dtype=torch.float32)
    c = c.repeat(-(-M // c.numel()))[:M] * -64.0
    x = c[:, None].expand(M, N).to(xt).contiguous()
    gamma, beta = rand((N,), F32, 1, 0.1, 1.0), rand((N,), F32, 2)
    r = nv.nvfp4_layernorm(x, gamma, beta, 1e-5, out_dtype=F32)
    assert torch.equal(r.mean, c)
    assert torch.equal(r.y, beta.expand(M, N))
    assert bool(((r.rstd.double() - 1e-5 ** -0.5).abs() <= 4 * U * 1e-5 ** -0.5).all())


@pytest.mark.parametrize("M,N", [(8, 1), (8, 64), (8, 1023), (8, 5120), (8, 33000), (700, 264), (700, 5120), (700, 9008),
                                 (700, 2731), (700, 12379)])
def test_layernorm_of_a_row_with_an_infinity(M, N):
    """Its mean is infinite, its y NaN throughout; no other row takes notice."""
    x = rand((M, N), BF, 10)
    x[5, N - 1], x[6, 0] = float("inf"), float("-inf")
    r = nv.nvfp4_layernorm(x)
    assert r.mean[5:7].tolist() == [float("inf"), float("-inf")] and bool(r.rstd[5:7].isnan().all())
    bad = r.y.isnan().all(1)
    assert bad.nonzero().flatten().tolist() == [5, 6] and bool(r.y[~bad].isfinite().all())


def test_layernorm_amax_of_rows_whose_squares_vanish():
    """eps = 0 and values whose squares are zero in fp32: rstd is Inf and so is every y.
    The amax is that of the outputs; the columns beside a row, which its vectors
    take along, are none (0 * Inf would make it NaN)."""
    for M, N, ld in ((700, 2000, 2000), (700, 2000, 2001), (700, 1538, 1539), (5, 2000, 2001), (700, 9008, 9009)):
        x = torch.full((M, N), 1e-30, device="cuda")
        x[:, ::2] *= -1
        xv = strided(x.to(BF), ld - N, 0)[1]
        r = nv.nvfp4_layernorm(xv, eps=0.0, out=strided(torch.zeros_like(xv), ld - N, 0)[1], want_amax=True)
        assert bool(r.y.isinf().all()) and r.amax.tolist() == [float("inf")] * 2, (M, N, ld)


def test_layernorm_statistics_of_empty_rows_are_nan():
    """The mean of no values is 0 / 0."""
    for M in (1, 3, 1000):
        junk = [torch.zeros(2 * M + 8, device="cuda") for _ in range(4)]  # memory that the results may be given
        del junk
        r = nv.nvfp4_layernorm(torch.empty((M, 0), dtype=BF, device="cuda"), want_amax=True)
        assert r.mean.shape == (M,) and bool(r.mean.isnan().all()) and bool(r.rstd.isnan().all())
        assert r.amax.tolist() == [0.0, 0.0]


# ---------------------------------------------------------------- erf GELU in fp32


def far(got, want):
    return float((got.double() - want).norm() / want.norm())


def linear_of(z, tokens):
    """nvfp4_linear's erf GELU of z: zero operands, z as the bias, the same in every token's row."""
    b = operand(z.numel(), 64, 3)
    a = (torch.zeros((tokens, 32), dtype=torch.uint8, device="cuda"),
         torch.zeros((-(-tokens // 128) * 128, 4), dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"))
    d = nv.nvfp4_linear(*a, *b, bias=z, act=nv.ACT_GELU, out_dtype=F32).d
    assert torch.equal(d[0].expand_as(d), d)
    return d[0]


# one and several tokens: joined pieces, whole tiles, pairs of SMs with vectors and with single values
GELU_PATHS = [(1, 20480), (40, 20480), (200, 640), (1100, 4096), (1100, 4097)]


@pytest.mark.parametrize("tokens,N", GELU_PATHS)
def test_gelu_in_fp32_is_as_close_as_the_plain_formula(tokens, N):
    """No farther from the 64-bit formula than z / 2 * (1 + erf(z / sqrt 2)) in
    elementary fp32 operations, by more than a quarter."""
    z = rand((N,), F32, 1, 1.5)
    plain = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    want = act64(z.double(), nv.ACT_GELU)
    assert far(linear_of(z, tokens), want) <= 1.25 * far(plain, want)


@pytest.mark.parametrize("M,N", [(64, 4096), (64, 4097), (1000, 1024), (1000, 1001)])
def test_gelu_gradient_in_fp32_is_as_close_as_the_plain_formula(M, N):
    z = rand((M, N), F32, 2, 1.5)
    plain = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    want = slope64(z.double(), nv.ACT_GELU)
    got = nv.nvfp4_act_backward(torch.ones_like(z), z, nv.ACT_GELU).dz
    assert far(got, want) <= 1.25 * far(plain, want)


def test_gelu_in_fp32_keeps_the_tail():
    """For z in [-5, -2] value and derivative are tiny and still have their leading
    digits.  erfc(-z / sqrt 2) changes by z^2 <= 25 times its argument's relative
    error, of two roundings: 50 u; erfc itself is within 4 units (8 u).  The
    density's exponent z^2 / 2 <= 12.5 has one rounding, the exponential is within 2
    units: 17 u.  Products add a few u.  In the derivative Phi + z phi the first
    term is at most a quarter of the second there, so that errors grow by at most
    1.25 / 0.75: all below 2^7 u."""
    z = torch.linspace(-5.0, -2.0, 20000, device="cuda")
    for got, want in ((linear_of(z, 1), act64(z.double(), nv.ACT_GELU)),
                      (linear_of(z, 1100), act64(z.double(), nv.ACT_GELU)),
                      (nv.nvfp4_act_backward(torch.ones_like(z)[None], z[None], nv.ACT_GELU).dz[0],
                       slope64(z.double(), nv.ACT_GELU))):
        assert float(((got.double() - want) / want).abs().max()) <= 2.0 ** 7 * U


@pytest.mark.parametrize("act", range(1, 5))
@pytest.mark.parametrize("tokens", [1, 40, 1100])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_activations_of_extreme_values(act, tokens, dt):
    """Large and tiny z have the limits of the activation, Inf stays, NaN stays; -Inf
    is 0 for ReLU and, as the formulas have it (-Inf * 0), NaN for the others."""
    z = torch.zeros(2600, device="cuda")
    z[:11] = torch.tensor([0.0, 1e-30, 1e30, -1e30, 1e4, -1e4, 30.0, -30.0, float("inf"), float("nan"), float("-inf")])
    b = operand(z.numel(), 64, 3)
    a = (torch.zeros((tokens, 32), dtype=torch.uint8, device="cuda"),
         torch.zeros((-(-tokens // 128) * 128, 4), dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"))
    r = nv.nvfp4_linear(*a, *b, bias=z, act=act, out_dtype=dt, want_z=True)
    assert torch.equal(r.z[0, :9], z[:9].to(dt))
    d = r.d[-1, :11].float()
    big = torch.tensor([1e30, 1e4, 30.0], device="cuda").to(dt).float()
    assert d[0] == 0 and 0 <= d[1] <= z[1].to(dt)
    assert torch.equal(d[[2, 4, 6]], big) and bool((d[[3, 5, 7]].abs() <= 1e-10).all())
    assert d[8] == float("inf") and bool(d[9].isnan())
    assert d[10] == 0 if act == nv.ACT_RELU else bool(d[10].isnan())
    assert bool((r.d[:, 11:] == 0).all())


# ---------------------------------------------------------------- scratch memory


GUARD = 4096


def guarded(n):
    """n bytes between guard bytes: (buffer, the n bytes)."""
    base = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return base, base[GUARD:GUARD + n]


def guards_hold(base):
    return bool((base[:GUARD] == 0xA5).all() and (base[-GUARD:] == 0xA5).all())


@pytest.mark.parametrize("M,N,pad", [(1, 1, 0), (1, 5120, 0), (1, 20480, 0), (2, 133, 0), (3, 5128, 0), (7, 33001, 0),
                                     (100, 2731, 0), (700, 5120, 0), (1217, 1001, 0), (1300, 4096, 0), (2000, 8192, 0),
                                     (900, 12288, 0), (16384, 264, 0), (3000, 333, 1)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_layernorm_backward_in_the_workspace_asked_for(M, N, pad, dt):
    """With exactly the bytes asked for: nothing beside them is written."""
    L = nv.layer_lib()
    x, dy, dres = rand((M, N), dt, M + N, 2.0, 0.3), rand((M, N), dt, M + N + 1, 1e-3), rand((M, N), dt, 14, 1e-3)
    mean, rstd = stats(x)
    n = L.nvfp4_layernorm_backward_workspace(M, N)
    for res in (None, dres):
        base, ws = guarded(n)
        xv, dyv = strided(x, pad, 0)[1], strided(dy, pad, 0)[1]
        dx, sums = strided(torch.zeros_like(x), pad, 0)[1], torch.empty((2, N), device="cuda")
        rv = strided(res, pad, 0)[1] if res is not None else None
        b = int(dt is BF)
        assert L.nvfp4_layernorm_backward(dyv.data_ptr(), N + pad, b, xv.data_ptr(), N + pad, b, M, N, mean.data_ptr(),
                                          rstd.data_ptr(), None, 0, rv.data_ptr() if rv is not None else None, N + pad,
                                          dx.data_ptr(), N + pad, sums[0].data_ptr(), sums[1].data_ptr(),
                                          ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
        check_norm_grad(dy, x, mean, rstd, None, res, nv.NormGrads(dx, sums[0], sums[1]))
        assert guards_hold(base)


@pytest.mark.parametrize("M,N,pad", [(1, 33, 0), (300, 33, 0), (700, 20480, 0), (513, 2048, 0), (4000, 1001, 0),
                                     (4001, 1002, 0), (4000, 1004, 0), (16384, 72, 1), (5000, 9, 0)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_act_backward_in_the_workspace_asked_for(M, N, pad, dt):
    L = nv.layer_lib()
    dy, z = rand((M, N), dt, M + N, 1e-3), rand((M, N), dt, N, 2.0)
    n = L.nvfp4_act_backward_workspace(M, N)
    base, ws = guarded(n)
    dyv, zv, dz = strided(dy, pad, 0)[1], strided(z, pad, 0)[1], strided(torch.zeros_like(z), pad, 0)[1]
    dbias = torch.empty(N, device="cuda")
    assert L.nvfp4_act_backward(dyv.data_ptr(), N + pad, zv.data_ptr(), N + pad, M, N, int(dt is BF), nv.ACT_SILU,
                                dz.data_ptr(), N + pad, dbias.data_ptr(), ws.data_ptr(), n,
                                torch.cuda.current_stream().cuda_stream) == 0
    check_act_grad(dy, z, nv.ACT_SILU, nv.ActGrads(dz, dbias))
    assert guards_hold(base)


# ---------------------------------------------------------------- long sums over rows


# A sum's first value is 2^24 and all others are 1, so that every one added to it alone is lost (2^24 + 1 is a tie,
# which goes to the even 2^24).  With chains of at most 512 values at most 511 are lost; what the join adds are multiples
# of 2 or lost too, one rounding of at most 1 for each of its additions.
MOST_LOST = 511 + 64


def first_dwarfs_the_rest(M, N, offset):
    base = torch.ones(offset + M * N, dtype=BF, device="cuda")
    t = base[offset:].view(M, N)
    t[0] = 2.0 ** 24
    return t


@pytest.mark.parametrize("M,N,offset", [(16384, 81920, 0), (16384, 40001, 0), (8192, 20481, 1), (1000000, 64, 0),
                                        (1000000, 33, 1)])
def test_bias_gradient_of_many_rows_loses_no_more_than_a_chain(M, N, offset):
    dy = first_dwarfs_the_rest(M, N, offset)
    got = nv.nvfp4_act_backward(dy, None, nv.ACT_NONE, want_dz=False).dbias
    assert float((got.double() - (2.0 ** 24 + M - 1)).abs().max()) <= MOST_LOST


@pytest.mark.parametrize("M,N,offset", [(1600000, 264, 0), (170000, 5120, 0), (170000, 5001, 1), (170000, 4999, 0),
                                        (400000, 1001, 1), (8192, 20481, 1), (16384, 81920, 0)])
def test_beta_gradient_of_many_rows_loses_no_more_than_a_chain(M, N, offset):
    dy = first_dwarfs_the_rest(M, N, offset)
    mean, rstd = torch.ones(M, device="cuda"), torch.ones(M, device="cuda")
    r = nv.nvfp4_layernorm_backward(dy, dy, mean, rstd)
    assert float((r.dbeta.double() - (2.0 ** 24 + M - 1)).abs().max()) <= MOST_LOST


# ---------------------------------------------------------------- shapes and outputs that nothing else reaches


@pytest.mark.parametrize("xt,dt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("M,N,pad", [(1300, 1, 0), (1301, 2, 0), (1300, 3, 0), (1217, 4, 1), (1300, 5, 0), (1299, 6, 0),
                                     (2001, 7, 0), (1300, 7, 2), (1300, 3, 6)])
def test_layernorm_backward_of_many_narrow_rows(M, N, pad, xt, dt):
    """A vector holds several rows: nothing beside a row is written, neighbours' NaN reaches no other."""
    x, dy, dres = rand((M, N), xt, M + N, 2.0, 0.3), rand((M, N), dt, M + N + 1, 1e-3), rand((M, N), xt, 14, 1e-3)
    gamma = rand((N,), F32, 13, 0.2, 1.0)
    mean, rstd = stats(x)
    base, out = strided(torch.zeros_like(x), pad, 0)
    xv, dyv, resv = strided(x, pad, 0)[1], strided(dy, pad, 0)[1], strided(dres, pad, 0)[1]
    r = nv.nvfp4_layernorm_backward(dyv, xv, mean, rstd, gamma, resv, out=out)
    check_norm_grad(dy, x, mean, rstd, gamma, dres, r)
    assert untouched(base, M, N, pad, 0)
    clean = r.dx.clone()
    xv[M // 2] = float("nan")
    got = nv.nvfp4_layernorm_backward(dyv, xv, mean, rstd, gamma, resv, out=resv).dx  # in place
    rows = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[rows], clean[rows])


@pytest.mark.parametrize("M,N,K", [(2050, 5001, 96), (2050, 5000, 544), (2560, 5120, 64), (40, 640, 512)])
def test_linear_amax_beside_a_residual(M, N, K):
    a, b, res = operand(M, K, M + K), operand(N, K, N + K), rand((M, N), BF, 5)
    for act in (nv.ACT_NONE, nv.ACT_SILU):
        for z in (False, True):
            r = nv.nvfp4_linear(*a, *b, act=act, residual=res, want_z=z, want_amax=True)
            check_linear(a, b, K, r, None, act, res)
            assert r.amax.tolist() == [float(r.d.float().abs().max())] * 2


@pytest.mark.parametrize("M,N,K", [(2327, 1246, 96), (700, 2601, 288), (2050, 5006, 64), (1100, 2607, 160), (300, 260, 512),
                                   (1, 333, 64), (40, 333, 64), (200, 333, 64)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_rows_that_end_inside_16_bytes(M, N, K, dt):
    """Rows that begin at 16 bytes and do not end there: what lies behind a row's last
    value is another tensor's, for d and for z."""
    L = nv.layer_lib()
    per = 16 // dt.itemsize
    pad = -N % per + per * (M % 2)
    a, b = operand(-(-M // 16) * 16, K, M), operand(-(-N // 16) * 16, K, N + K, 0.05)
    a, b = (a[0][:M].contiguous(), a[1], a[2]), (b[0][:N].contiguous(), b[1], b[2])
    bias, res = rand((N,), F32, 3), rand((M, N), dt, 5)
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(max(16, L.nvfp4_linear_workspace(M, N, K)), dtype=torch.uint8, device="cuda")
    for r, keep in ((None, False), (None, True), (res, False), (res, True)):
        d_base, d = strided(r if r is not None else torch.zeros((M, N), dtype=dt, device="cuda"), pad, 0)
        z_base, z = strided(torch.zeros((M, N), dtype=dt, device="cuda"), pad, 0)
        amax = torch.empty(2, device="cuda")
        assert L.nvfp4_linear(*[t.data_ptr() for t in (*a, *b)], M, N, K, bias.data_ptr(), 0, nv.ACT_SILU,
                              d.data_ptr() if r is not None else None, N + pad, z.data_ptr() if keep else None, N + pad,
                              d.data_ptr(), N + pad, int(dt is BF), amax.data_ptr(), ws.data_ptr(), ws.numel(), None,
                              s) == 0
        check_linear(a, b, K, nv.LinearOut(d, z if keep else None, amax), bias, nv.ACT_SILU, r, dt)
        assert untouched(d_base, M, N, pad, 0) and untouched(z_base, M, N, pad, 0)
        assert amax.tolist() == [float(d.float().abs().max())] * 2
