"""The attention operators where they are easily wrong: sizes of scores, weights and queries far apart,
long contexts, infinities beside what passes.

Tolerances.  A score is held to d = 2^-16 of sum |q k| |scale|, as in test_gpu_attention.py.  A
weight is rounded to fp16 where it meets the values: 2^-11 of itself, or half of fp16's smallest
step, 2^-25, where it is small; the row's largest stands there at 2^7 or above, so that this is
2^-32 of it, whatever the number of keys.  With the exponential (2^-14) o is held to
u |o| + (2^-11 + 2^-14 + 2 d) sum w |v| + 2^-32 sum |v| / sum exp(s - max), u = 2^-8 for bf16.
"""
import ctypes
import math
import threading

import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300.attention import Batch, Cache, Tokens
from nvfp4_bit_block_gb300.build import build_attention_selftest
from attention_oracle import rope64, sequence64, visible
from test_gpu_attention import (BF, F32, T_SCORE, T_WEIGHT, U_OUT, Work, both_kernels, built, check_rope_grad, company, freqs, gen, ints,  # noqa: F401
                                placed, rand, within)

pytestmark = pytest.mark.gpu
T_SMALL = 2.0 ** -32


def check(w, q, r, scale=None, causal=True, window=0, sinks=0):
    """o and lse of every row of the batch against the formula in 64 bits."""
    scale = w.dim ** -0.5 if scale is None else scale
    G = q.shape[1] // w.heads
    at = 0
    for b, (n, m) in enumerate(zip(w.lens, w.news)):
        if m == 0:
            continue
        k, v = (t.transpose(0, 1) for t in sequence64(w.cache, w.table, b, n))  # heads, keys, values
        see = visible(n, m, causal, window, sinks, q.device)
        for h in range(q.shape[1]):
            x, kh, vh = q[at:at + m, h].double(), k[h // G], v[h // G]
            s = (x @ kh.t() * scale).masked_fill(~see, -math.inf)
            top = s.amax(-1, keepdim=True).clamp(min=-1e300)
            e = torch.exp(s - top)
            total = e.sum(-1, keepdim=True)
            d = T_SCORE * (x.abs() @ kh.abs().t() * abs(scale)).masked_fill(~see, 0.0).amax(-1, keepdim=True)
            some = total > 0
            total = torch.where(some, total, torch.ones_like(total))
            o, lse = e @ vh / total, torch.where(some, top + total.log(), torch.full_like(top, -math.inf))
            bar = U_OUT[BF] * o.abs() + (T_WEIGHT + 2 * d) * (e @ vh.abs() / total) + T_SMALL * (see.double() @ vh.abs() / total)
            within(r.o[at:at + m, h], o, bar, f"o, sequence {b}, head {h}")
            if r.lse is not None:
                within(r.lse[at:at + m, h], lse[:, 0], (d + 2.0 ** -17 + 2.0 ** -23 * lse.abs().nan_to_num(0.0, posinf=0.0))[:, 0],
                       f"lse, sequence {b}, head {h}")
        at += m


def attend(w, q, **kw):
    st = ints([0])
    r = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True, status=st, **kw)
    assert st.item() == 0
    check(w, q, r, **kw)
    return r


def put(w, k, v):
    """Keys and values of every position of every sequence."""
    starts = [0]
    for n in w.lens:
        starts.append(starts[-1] + n)
    nv.nvfp4_cache_write(k, v, w.cache, ints(starts), w.lengths, w.table)


# ---------------------------------------------------------------- attention


@both_kernels
@pytest.mark.parametrize("gap", [8.0, 11.0, 13.5, 15.0, 17.0])
@pytest.mark.parametrize("B,n,m,dim", [(16, 2048, 40, 64), (2, 9000, 40, 128), (3, 2500, 1, 256), (160, 900, 1, 32)])
def test_one_key_outweighs_the_others(B, n, m, dim, gap):
    """The first key's score lies `gap` above all others and its value is zero: the result is made of weights that are
    e^-gap of the largest."""
    w = Work([n - 7 * b % 300 for b in range(B)], [m] * B, 8 if B < 100 else 2, dim, 16, (2.0 ** -5, 2.0 ** -5), seed=1)
    k = torch.zeros((sum(w.lens), w.heads, dim), device="cuda")
    v = 1 + 0.25 * rand(k.shape, F32, 2)
    at = 0
    for length in w.lens:
        k[at, :, 0] = 6.0
        v[at] = 0.0
        at += length
    put(w, k, v)
    q = rand((w.T, w.heads, dim), BF, 3)
    q[..., 0] = gap / 6
    attend(w, q, scale=1.0)


SHAPES = [([300, 64, 1], [1, 1, 1], 2, 5, 128, 16), ([150, 90], [9, 30], 1, 3, 64, 16), ([270, 130], [200, 130], 2, 2, 96, 32),
          ([400], [333], 1, 3, 256, 64)]


@both_kernels
@pytest.mark.parametrize("scale", [0.3, -0.2, 1.7, 0.0, -0.0, 1e-6, -1e-30, 1e-38, 2.0 ** -149])
@pytest.mark.parametrize("lens,news,heads,group,dim,page", SHAPES)
def test_scales(lens, news, heads, group, dim, page, scale):
    """Any factor of the scores: negative ones, none, and those that vanish; hidden keys stay hidden."""
    w = Work(lens, news, heads, dim, page, seed=4)
    w.fill()
    q = rand((w.T, heads * group, dim), BF, 5)
    attend(w, q, scale=scale)
    attend(w, q, scale=scale, causal=False)
    attend(w, q, scale=scale, window=37, sinks=5)


@both_kernels
@pytest.mark.parametrize("news", [[1, 1], [9, 30], [150, 180]])
def test_scores_beyond_what_a_float_resolves(news):
    """Scores of 2^20 and far more that differ by a few: whatever is left of their differences, the weights are none
    that a sum of ones would show."""
    w = Work([1500, 700], news, 1, 64, 16, (2.0 ** -5, 2.0 ** -5), seed=6)
    k = torch.zeros((sum(w.lens), 1, 64), device="cuda")
    k[..., 0] = 6.0
    near = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0], device="cuda")
    put(w, k, torch.ones_like(k))
    held = sequence64(w.cache, w.table, 0, 1)[1]  # what the cache has for 1, the same everywhere
    for p in range(18, 100, 3):
        k[..., 16] = near[torch.randint(0, 6, (sum(w.lens),), generator=gen(p), device="cuda")][:, None]
        put(w, k, torch.ones_like(k))
        q = torch.zeros((w.T, 3, 64), device="cuda")
        q[..., 0] = torch.tensor([1.0, -1.5, 1.25], device="cuda") * 2.0 ** p
        q[..., 16] = torch.tensor([1.0, 2.0, 4.0], device="cuda")
        for f in (1.0, 2.0 ** min(p - 24, 8)):
            q[..., 16] *= f
            r = nv.nvfp4_cache_attention(q.to(BF), w.cache, *w.batch, scale=1.0, want_lse=True)
            within(r.o, held.expand(r.o.shape), (U_OUT[BF] + T_WEIGHT) * held, f"2^{p}")
            want = q[:, :, 0].double() * 6
            within(r.lse, want, 2.0 ** -21 * want.abs() + 24 * q[..., 16].double() + 20, f"lse, 2^{p}")


@both_kernels
@pytest.mark.parametrize("news", [[1, 1], [9, 30], [150, 180]])
@pytest.mark.parametrize("down", [10, 17, 22, 27])
def test_queries_whose_values_lie_far_apart(news, down):
    """A query's largest value meets zeros only: the scores are those of values 2^-down of it, which keep their digits."""
    w = Work([400, 200], news, 2, 64, 16, seed=7)
    k, v = rand((600, 2, 64), F32, 8), rand((600, 2, 64), F32, 9)
    k[..., :16] = 0.0
    put(w, k, v)
    for size in (1.0, 2.0 ** 100, 2.0 ** -90):
        q = rand((w.T, 6, 64), F32, 10) * size
        q[..., 3] = 2.0 ** down * size
        attend(w, q.to(BF), scale=0.125 / size)


@both_kernels
@pytest.mark.parametrize("lens,news,group,dim", [([100000, 5, 40000], [1, 1, 2], 4, 64), ([100000], [40], 2, 64),
                                                 ([30000, 20000], [70, 1], 1, 128)])
def test_long_contexts_with_few_keys_that_count(lens, news, group, dim):
    """The weight sits on some forty keys, all along each sequence: none of its pieces can be lost or counted twice."""
    w = Work(lens, news, 1, dim, 64, (2.0 ** -5, 2.0 ** -6), seed=11)
    k, v = 0.1 * rand((sum(lens), 1, dim), F32, 12), rand((sum(lens), 1, dim), F32, 13)
    at = 0
    for n in lens:
        for i in torch.linspace(0, max(n - max(news) - 1, 0), min(n, 41)).long().unique().tolist():
            k[at + i, 0, 0] = 6.0
        at += n
    put(w, k, v)
    q = rand((w.T, group, dim), BF, 14)
    q[..., 0] = 3.0
    attend(w, q, scale=1.0)


def test_heads_that_lie_far_apart():
    """Heads first, 2^32 bytes and more from one to the next."""
    H, D = 3, 128
    w = Work([200, 90], [70, 1], H, D, 64, seed=18, order="hpsd")
    w.fill()

    def apart(t, step):
        P, H, S, n = t.shape
        base = torch.empty((H - 1) * step + P * S * n, dtype=torch.uint8, device="cuda")
        v = base.as_strided((P, H, S, n), (S * n, step, n, 1))
        v.copy_(t)
        return v
    c = w.cache
    far = nv.KVCache(apart(c.k_codes, 2 ** 32 + 4096), apart(c.k_scales, 2 ** 31 + 1024), apart(c.v_codes, 2 ** 32 + 4096),
                     apart(c.v_scales, 2 ** 31 + 1024), c.alpha)
    q = rand((w.T, 2 * H, D), BF, 19)
    for batch in (w.batch, (w.starts[1:] - w.starts[1], w.lengths[1:], w.table[1:])):
        m = int(batch[0][-1])
        want, got = (nv.nvfp4_cache_attention(q[:m], x, *batch, want_lse=True) for x in (c, far))
        assert torch.equal(got.o, want.o) and torch.equal(got.lse, want.lse)
        a, b = (nv.nvfp4_cache_read(x, *batch, tokens=m) for x in (c, far))
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    k, v = rand((w.T, H, D), BF, 20), rand((w.T, H, D), BF, 21)
    for x in (c, far):
        nv.nvfp4_cache_write(k, v, x, *w.batch)
    assert all(torch.equal(a, b) for a, b in zip(c.tensors(), far.tensors()))


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 31 - 65])
@pytest.mark.parametrize("window,sinks", [(1, 2 ** 31 - 1), (40, 2 ** 31 - 70), (2 ** 31 - 1, 5), (100, 100)])
def test_the_longest_contexts(length, window, sinks):
    """Positions up to the last that 32 bits hold, on one page again and again.  2^31 equal rounds of the page's weights
    are summed in fp32, at most 2^17 of them one after another in a lane (2^27 chunks of 16 keys in 4 x 760 warps):
    off by 2^-7 where the roundings all go one way."""
    page, D = 65536, 32
    w = Work([page], [1], 1, D, page, seed=25)
    w.fill()
    q = rand((1, 2, D), BF, 26)
    table = w.table[:, :1].expand(1, 32768).contiguous()
    st = ints([0])
    r = nv.nvfp4_cache_attention(q, w.cache, w.starts, ints([length]), table, window=window, sinks=sinks, want_lse=True, status=st)
    assert st.item() == 0
    k, v = (t[:, 0] for t in sequence64(w.cache, w.table, 0, page))
    # how often each of the page's keys is visible
    often = torch.zeros(page, dtype=torch.float64, device="cuda")

    def count(a, b):  # positions a .. b - 1
        if b <= a:
            return
        first, last = a // page, (b - 1) // page
        if first == last:
            often[a % page:(b - 1) % page + 1] += 1
        else:
            often[a % page:] += 1
            often[:(b - 1) % page + 1] += 1
            often.add_(last - first - 1)
    low = max(0, length - window)
    count(low, length)
    count(0, min(sinks, low))
    s = q[0].double() @ k.t() * D ** -0.5
    e = torch.exp(s - s.amax(-1, keepdim=True)) * often
    total = e.sum(-1, keepdim=True)
    long = 2.0 ** -7 if length - low + min(sinks, low) > 2 ** 20 else 0.0
    o = e @ v / total
    within(r.o[0], o, U_OUT[BF] * o.abs() + (T_WEIGHT + 2.0 ** -12 + 2 * long) * (e @ v.abs() / total), "o")
    within(r.lse[0], (s.amax(-1, keepdim=True) + total.log())[:, 0], 2.0 ** -13 + long, "lse")


@pytest.mark.parametrize("n,m,dim", [(900, 200, 128), (321, 300, 256)])
def test_blocks_that_give_up_with_products_behind_them(n, m, dim):
    """A build whose keys stop coming after four blocks: what was issued is waited for before the tensor memory is freed,
    and the calls behind it, one of them another user of that memory, have all of it."""
    L = ctypes.CDLL(build_attention_selftest())
    w = Work([n], [m], 2, dim, 16, seed=22)
    w.fill()
    q, st = rand((m, 4, dim), BF, 23), ints([0])
    o, p, c = torch.zeros_like(q), ctypes.c_void_p, w.cache
    flags = nv.ROWWISE | nv.SF_SWIZZLED
    x = rand((300, 256), BF, 24)
    z = nv.nvfp4_quantize(x, nv.nvfp4_amax(x, flags), flags)
    linear = lambda: nv.nvfp4_linear(z.q_row, z.s_row, z.alpha[0:1], z.q_row, z.s_row, z.alpha[0:1]).d
    want = linear().clone()
    args = [p(t.data_ptr()) for t in (q, o, c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.alpha, w.starts, w.lengths, w.table)]
    torch.cuda.synchronize()
    assert L.nvfp4_selftest_attend_many(*args, m, 2, 2, dim, 16, w.table.shape[1], p(st.data_ptr())) == 0
    d = linear()
    assert st.item() == -8 and torch.equal(d, want)
    check(w, q, nv.nvfp4_cache_attention(q, c, *w.batch, want_lse=True))


@both_kernels
@pytest.mark.parametrize("lens,news,heads,group,dim", [([300], [1], 1, 5000, 32), ([90, 33], [2, 1], 1, 1500, 64),
                                                       ([40], [3], 300, 2, 32), ([17, 5, 0], [1, 1, 0], 3000, 1, 32)])
def test_very_many_heads(lens, news, heads, group, dim):
    w = Work(lens, news, heads, dim, 16, seed=32)
    w.fill()
    q = rand((w.T, heads * group, dim), BF, 33)
    r = attend(w, q)
    again = nv.nvfp4_cache_attention(q, w.cache, *w.batch, want_lse=True)
    assert torch.equal(again.o, r.o) and torch.equal(again.lse, r.lse)


def spread(t, step):
    """t (T, H, D) with `step` elements from token to token."""
    T, H, D = t.shape
    v = torch.empty((T - 1) * step + H * D, dtype=t.dtype, device="cuda").as_strided((T, H, D), (step, D, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("m", [2, 3])
def test_tokens_that_lie_far_apart(m):
    """2^31 elements and more from token to token, of queries, keys, values and results of each call."""
    step, H, D = 2 ** 31 + 64, 2, 64
    w = Work([40 + m], [m], H, D, 16, seed=34)
    w.fill()
    q, k, v = (rand((m, h, D), BF, 35 + h) for h in (20, H, H))
    pos, f = torch.arange(40, 40 + m, device="cuda", dtype=torch.int32), freqs(32)
    a = nv.nvfp4_qk_rope(q, k, pos, f)
    b = nv.nvfp4_qk_rope(spread(q, step), k, pos, f, out_q=spread(q, step))
    assert torch.equal(a.q, b.q) and torch.equal(a.k, b.k)
    far = b.q
    ga = nv.nvfp4_qk_rope_backward(q, k, a.q, a.k, pos, f)
    gb = nv.nvfp4_qk_rope_backward(q, k, far, a.k, pos, f, out_q=far)
    assert torch.equal(ga.dq, gb.dq) and torch.equal(ga.dgamma_q, gb.dgamma_q)
    del far, b, gb
    nv.nvfp4_cache_write(k, v, w.cache, *w.batch)
    before = [t.clone() for t in w.cache.tensors()]
    far = spread(v, step)
    w.cache.v_codes.zero_()
    nv.nvfp4_cache_write(k, far, w.cache, *w.batch)
    pages, rows = (torch.tensor(x, device="cuda") for x in zip(*w.slots()))
    assert torch.equal(w.cache.v_codes[pages, :, rows], before[2][pages, :, rows])
    far.zero_()
    r = nv.nvfp4_cache_read(w.cache, *w.batch, out_v=far, want_k=False)
    assert torch.equal(r.v, nv.nvfp4_cache_read(w.cache, *w.batch, tokens=m).v)
    del far, r
    w.cache.v_codes.copy_(before[2])
    o = attend(w, q).o
    far = spread(q, step)
    assert torch.equal(nv.nvfp4_cache_attention(far, w.cache, *w.batch, out=far).o, o)


def test_host_threads_at_once():
    """C callers launch from several threads, heads of different sizes, few rows and many; no thread's launch may depend on
    what another has just asked for."""
    L = nv.attention_lib()
    jobs, faults = [], []
    for i, (dim, news) in enumerate([(64, [1, 1]), (128, [3, 2]), (256, [1, 4]), (96, [90, 70]), (128, [150, 200]), (256, [80, 1])]):
        w = Work([300, 210], news, 2, dim, 16, seed=40 + i)
        w.fill()
        q = rand((w.T, 8, dim), BF, 50 + i)
        want = nv.nvfp4_cache_attention(q, w.cache, *w.batch).o
        c, kc, sc = w.cache, w.cache.k_codes, w.cache.k_scales
        cache = Cache(c.k_codes.data_ptr(), c.k_scales.data_ptr(), c.v_codes.data_ptr(), c.v_scales.data_ptr(), c.alpha.data_ptr(),
                      kc.shape[0], 2, 16, dim, *kc.stride()[:3], *sc.stride()[:3])
        batch = Batch(w.starts.data_ptr(), w.lengths.data_ptr(), w.table.data_ptr(), 2, w.table.shape[1], w.table.stride(0))
        n = L.nvfp4_cache_attention_workspace(w.T, 8, 2, dim, 2)
        ws, o = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(q)
        tq, to = (Tokens(t.data_ptr(), t.stride(0), t.stride(1)) for t in (q, o))
        jobs.append((lambda s, tq=tq, to=to, w=w, cache=cache, batch=batch, ws=ws, n=n, dim=dim, q=q: L.nvfp4_cache_attention(
            ctypes.byref(tq), w.T, 8, ctypes.byref(cache), ctypes.byref(batch), dim ** -0.5, 1, 0, 0, ctypes.byref(to), None,
            ws.data_ptr(), n, None, s), o, want))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(call):
        s = torch.cuda.Stream()
        start.wait()
        for _ in range(200):
            if status := call(s.cuda_stream):
                faults.append(status)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(j[0],)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not faults
    for _, o, want in jobs:
        assert torch.equal(o, want)


# ---------------------------------------------------------------- norm and rotation


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("D,R,tp,hp,off", [(128, 32, 0, 0, 0), (96, 24, 4, 4, 4), (64, 10, 2, 2, 2), (66, 9, 1, 1, 1),
                                           (128, 0, 0, 0, 0), (34, 17, 0, 0, 0)])
def test_what_passes_is_what_came(D, R, tp, hp, off, xt, yt, inter):
    """Values outside the rotated part come out as they went in, infinities and NaN beside them or not; in the rotated
    part such a value reaches its pair alone."""
    T, H = 5, 3
    x = rand((T, H, D), xt, 15)
    odd = [float("inf"), float("nan"), float("-inf")]
    for t in range(T):
        for h in range(H):
            for c in range(2 * R, D, 5 + t):
                x[t, h, c] = odd[(t + h + c) % 3]
    if R:
        x[1, 1, 1 if inter else 0] = float("inf")
        x[2, 0, 2 * R - 1] = float("nan")
    pos, f = ints([0, 1, 7, 900, 123456]), freqs(R)
    q = placed(x, tp, hp, off)[1]
    out = placed(torch.zeros((T, H, D), dtype=yt, device="cuda"), tp, hp, off)[1]
    for back in (False, True):
        if back:
            got = nv.nvfp4_qk_rope_backward(q, q, None, None, pos, f, norm=False, interleaved=inter,
                                            out_q=out if xt is yt else None).dq
            turn = -f
        else:
            got = nv.nvfp4_qk_rope(q, q, pos, f, norm=False, interleaved=inter, out_q=out, out_dtype=yt).q
            turn = f
        want = x[..., 2 * R:].to(got.dtype)
        passed = got[..., 2 * R:]
        assert bool(((passed == want) | (passed.isnan() & want.isnan())).all())
        clean = torch.where(x.isfinite(), x, torch.zeros_like(x))
        ref, size = rope64(clean, pos, turn, None, 0, False, inter)
        keep = torch.ones((T, H, D), dtype=torch.bool, device="cuda")
        keep[..., 2 * R:] = False
        if R:
            for t, h, i in ((1, 1, 0), (2, 0, R - 1)):
                keep[t, h, (2 * i if inter else i)] = keep[t, h, (2 * i + 1 if inter else i + R)] = False
        within(got[keep], ref[keep], U_OUT[got.dtype] * ref[keep].abs() + 2.0 ** -18 * size[keep], "turned")


@pytest.mark.parametrize("D,R,hp", [(128, 32, 0), (96, 24, 1), (64, 10, 2)])
def test_an_infinite_gradient_reaches_its_own_weight_alone(D, R, hp):
    """Of the gradient of the norm's weights, where what passes holds an infinity."""
    T, H = 9, 2
    x, dy = placed(rand((T, H, D), F32, 16), 0, hp, 0)[1], placed(rand((T, H, D), F32, 17), 0, hp, 0)[1]
    pos, f = torch.arange(T, device="cuda", dtype=torch.int32), freqs(R)
    want = nv.nvfp4_qk_rope_backward(dy, dy, x, x, pos, f).dgamma_q
    for c in (2 * R, D - 1):
        odd = dy.clone()
        odd[4, 1, c] = float("inf")
        odd = placed(odd, 0, hp, 0)[1]
        got = nv.nvfp4_qk_rope_backward(odd, dy, x, x, pos, f).dgamma_q
        assert bool(got[c].isinf())
        got[c] = want[c]
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [151, 152, 153, 304, 305, 515, 608, 609, 1216, 1217])
def test_gradients_where_blocks_take_more_tokens(T):
    """Numbers of tokens around those at which a block takes two, four and eight; guard bytes around a workspace of exactly
    the size that the C ABI asks for."""
    Hq, Hk, D, R = 5, 2, 64, 32
    q, k, dq, dk = (rand((T, h, D), F32, 27 + i) for i, h in enumerate((Hq, Hk, Hq, Hk)))
    g, pos, f = rand((D,), F32, 31, 0.2, 1.0), torch.arange(T, device="cuda", dtype=torch.int32), freqs(R)
    r = nv.nvfp4_qk_rope_backward(dq, dk, q, k, pos, f, g, g)
    check_rope_grad(dq, q, r.dq, r.dgamma_q, pos, f, g, 1e-6, True, False, "q")
    check_rope_grad(dk, k, r.dk, r.dgamma_k, pos, f, g, 1e-6, True, False, "k")
    L = nv.attention_lib()
    n = L.nvfp4_qk_rope_backward_workspace(T, Hq, Hk, D)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    oq, ok, gq, gk = torch.empty_like(q), torch.empty_like(k), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    tok = lambda t: ctypes.byref(Tokens(t.data_ptr(), t.stride(0), t.stride(1)))
    assert L.nvfp4_qk_rope_backward(tok(dq), tok(dk), 0, tok(q), tok(k), 0, T, Hq, Hk, D, R, 0, pos.data_ptr(), f.data_ptr(), 1,
                                    1e-6, g.data_ptr(), g.data_ptr(), 0, tok(oq), tok(ok), gq.data_ptr(), gk.data_ptr(),
                                    ws.data_ptr() + 256, n, torch.cuda.current_stream().cuda_stream) == 0
    for a, b in ((oq, r.dq), (ok, r.dk), (gq, r.dgamma_q), (gk, r.dgamma_k)):
        assert torch.equal(a, b)
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + n:] == 0xA5).all())
