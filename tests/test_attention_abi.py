"""The C ABI of the attention operators (include/nvfp4_attention.h): the library exports what
the header declares and rejects bad arguments on the host (no GPU needed: these calls return
before any CUDA work is enqueued)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300 import attention
from nvfp4_bit_block_gb300.attention import Batch, Cache, Tokens
from nvfp4_bit_block_gb300.build import ATTENTION_LIB

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000  # fake aligned device addresses: never dereferenced
OK, NULL, SHAPE, ALIGN, FLAGS, CUDA = 0, -1, -2, -3, -4, -5
ref = ctypes.byref


@pytest.fixture(scope="module")
def L():
    nv.build()
    return nv.attention_lib()


def header():
    with open(os.path.join(ROOT, "include", "nvfp4_attention.h")) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_library_exports_exactly_the_declared_entry_points(L):
    declared = sorted(re.findall(r"NVFP4_API\s+(?:int|int64_t)\s+(nvfp4_\w+)\s*\(", header()))
    out = subprocess.run(["nm", "-D", "--defined-only", ATTENTION_LIB], capture_output=True, text=True).stdout
    assert sorted(set(re.findall(r"\bT (nvfp4_\w+)", out))) == declared
    for name in declared:
        assert name.endswith("_workspace") or callable(getattr(nv, name))


def test_header_is_plain_c_and_the_structures_match(tmp_path):
    src = tmp_path / "t.c"
    fields = {"nvfp4_tokens": Tokens, "nvfp4_kv_cache": Cache, "nvfp4_batch": Batch}
    lines = [f'printf("{n} %zu\\n", sizeof({n}));' for n in fields]
    lines += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for n, c in fields.items() for f, _ in c._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "nvfp4_attention.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0; }\n")
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                        str(tmp_path / "t")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = dict(line.split() for line in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.splitlines())
    for n, c in fields.items():
        assert int(out[n]) == ctypes.sizeof(c)
        for f, _ in c._fields_:
            assert int(out[f"{n}.{f}"]) == getattr(c, f).offset


def test_argument_counts_match_the_header(L):
    for name, args in re.findall(r"NVFP4_API\s+\w+\s+(nvfp4_\w+)\s*\((.*?)\)\s*;", header(), flags=re.S):
        kinds = [ctypes.c_void_p if "*" in x else {"int64_t": ctypes.c_int64, "int": ctypes.c_int,
                                                   "float": ctypes.c_float}[x.split()[0]] for x in args.split(",")]
        assert list(getattr(L, name).argtypes) == kinds, name


def tok(p, ts=256, hs=64):
    return Tokens(p, ts, hs)


def rope(L, **k):
    a = dict(q=tok(A), k=tok(B), xb=1, T=4, Hq=4, Hk=2, D=64, R=32, inter=0, pos=D, freq=D, norm=1, eps=1e-6, gq=D, gk=D,
             wb=0, oq=tok(C), ok=tok(C), yb=1)
    a.update(k)
    return L.nvfp4_qk_rope(*[ref(v) if isinstance(v, Tokens) else v for v in a.values()], None)


def test_rope_rejects_bad_arguments(L):
    assert rope(L, T=-1) == SHAPE and rope(L, T=2 ** 31) == SHAPE
    for bad in (dict(D=0), dict(D=63, R=0), dict(D=514), dict(R=33), dict(R=-1), dict(Hq=-1), dict(Hk=65536)):
        assert rope(L, **bad) == SHAPE, bad
    assert rope(L, q=tok(A, -1)) == SHAPE and rope(L, ok=tok(C, 256, 2 ** 62)) == SHAPE
    for p in ("q", "k", "oq", "ok", "pos", "freq"):
        assert rope(L, **{p: None}) == NULL, p
    assert rope(L, q=tok(None)) == NULL and rope(L, ok=tok(None)) == NULL
    assert rope(L, eps=-1.0) == FLAGS and rope(L, eps=float("nan")) == FLAGS and rope(L, norm=0) == FLAGS
    assert rope(L, q=tok(A + 1)) == ALIGN and rope(L, xb=0, k=tok(B + 2)) == ALIGN and rope(L, oq=tok(C + 1)) == ALIGN
    assert rope(L, pos=D + 2) == ALIGN and rope(L, freq=D + 1) == ALIGN and rope(L, gq=D + 2) == ALIGN
    assert rope(L, T=0, q=tok(None)) == OK and rope(L, Hq=0, Hk=0) == OK


def grad(L, **k):
    a = dict(dq=tok(A), dk=tok(B), yb=1, q=tok(A), k=tok(B), xb=1, T=4, Hq=4, Hk=2, D=64, R=32, inter=0, pos=D, freq=D,
             norm=1, eps=1e-6, gq=D, gk=D, wb=0, oq=tok(C), ok=tok(C), dgq=D, dgk=D, ws=A, wn=1 << 40)
    a.update(k)
    return L.nvfp4_qk_rope_backward(*[ref(v) if isinstance(v, Tokens) else v for v in a.values()], None)


def test_rope_backward_rejects_bad_arguments(L):
    assert grad(L, T=-1) == SHAPE and grad(L, D=513) == SHAPE and grad(L, R=40) == SHAPE
    for p in ("dq", "dk", "q", "k", "oq", "ok", "pos", "freq", "ws"):
        assert grad(L, **{p: None}) == NULL, p
    assert grad(L, norm=0, gq=None, gk=None) == FLAGS  # gradients of weights that are not there
    assert grad(L, dgq=D + 2) == ALIGN and grad(L, ws=A + 4) == ALIGN and grad(L, dq=tok(A + 1)) == ALIGN
    n = L.nvfp4_qk_rope_backward_workspace(4, 4, 2, 64)
    assert n > 0 and grad(L, wn=n - 1) == SHAPE
    assert L.nvfp4_qk_rope_backward_workspace(-1, 4, 2, 64) == SHAPE and L.nvfp4_qk_rope_backward_workspace(0, 4, 2, 64) == 0
    assert grad(L, T=0, dgq=None, dgk=None) == OK


@pytest.mark.parametrize("T", [1, 7, 1000, 16384, 10 ** 6, 2 ** 31 - 1])
def test_the_rope_gradients_workspace_stays_bounded(L, T):
    n = L.nvfp4_qk_rope_backward_workspace(T, 40, 8, 128)
    assert 0 < n <= (152 * 8 + T * 40 / 8 / 500 + 1) * 2 * 128 * 4


def cache(**k):
    a = dict(k_codes=A, k_scales=B, v_codes=A, v_scales=B, alpha_dev=D, pages=10, heads=2, page_size=16, dim=64,
             code_page=1024, code_head=512, code_row=32, scale_page=128, scale_head=64, scale_row=4)
    a.update(k)
    return Cache(*a.values())


def batch(**k):
    a = dict(starts=D, lengths=D, table=D, sequences=3, table_width=5, table_stride=5)
    a.update(k)
    return Batch(*a.values())


def write(L, f="nvfp4_cache_write", c={}, b={}, **k):
    a = dict(k=tok(A, 128), v=tok(B, 128), xb=1, T=4, cache=cache(**c), batch=batch(**b), status=None)
    a.update(k)
    return getattr(L, f)(*[ref(v) if isinstance(v, ctypes.Structure) else v for v in a.values()], None)


def attend(L, c={}, b={}, **k):
    a = dict(q=tok(A), T=4, Hq=4, cache=cache(**c), batch=batch(**b), scale=0.125, causal=1, window=0, sinks=0, o=tok(C),
             lse=None, ws=A, wn=1 << 40, status=None)
    a.update(k)
    return L.nvfp4_cache_attention(*[ref(v) if isinstance(v, ctypes.Structure) else v for v in a.values()], None)


@pytest.mark.parametrize("call", ["nvfp4_cache_write", "nvfp4_cache_read", "attend"])
def test_the_cache_and_the_batch_are_checked(L, call):
    f = (lambda **k: attend(L, **k)) if call == "attend" else (lambda **k: write(L, call, **k))
    for bad in (dict(pages=-1), dict(pages=2 ** 31), dict(heads=0), dict(page_size=8), dict(page_size=24), dict(dim=48),
                dict(dim=288), dict(dim=0), dict(code_row=16), dict(code_head=496), dict(code_page=1008),
                dict(scale_row=2), dict(scale_head=62), dict(scale_page=126), dict(code_page=0), dict(code_row=-32),
                dict(page_size=131072)):
        assert f(c=bad) == SHAPE, bad
    for bad in (dict(code_row=40, code_head=640, code_page=1280), dict(k_codes=A + 8), dict(v_codes=A + 4),
                dict(v_scales=B + 1), dict(alpha_dev=D + 2), dict(scale_row=5, scale_head=80, scale_page=160)):
        assert f(c=bad) == ALIGN, bad
    # rows before heads, heads before pages, a cache of one page
    assert f(c=dict(code_head=32, code_row=64, scale_head=4, scale_row=8), T=0) == OK
    assert f(c=dict(code_head=10 * 512, code_page=512, scale_head=640, scale_page=64), T=0) == OK
    assert f(c=dict(pages=1, code_page=0, scale_page=0), T=0) == OK
    for bad in (dict(sequences=-1), dict(table_width=-1), dict(table_stride=-1), dict(table_width=2 ** 31)):
        assert f(b=bad) == SHAPE, bad
    for bad in (dict(starts=None), dict(lengths=None), dict(table=None)):
        assert f(b=bad) == NULL, bad
    for bad in (dict(k_codes=None), dict(v_scales=None), dict(alpha_dev=None)):
        assert f(c=bad) == NULL, bad
    assert f(cache=None) == NULL and f(batch=None) == NULL
    assert f(b=dict(starts=D + 2)) == ALIGN and f(status=D + 1) == ALIGN
    assert f(T=-1) == SHAPE and f(T=2 ** 31) == SHAPE
    assert f(T=0) == OK and f(b=dict(sequences=0)) == OK


def test_write_and_read_reject_bad_tokens(L):
    assert write(L, k=tok(None)) == NULL and write(L, v=None) == NULL
    assert write(L, k=tok(A, -1)) == SHAPE and write(L, v=tok(B + 1, 128)) == ALIGN and write(L, xb=0, k=tok(A + 2, 128)) == ALIGN
    r = lambda **k: write(L, "nvfp4_cache_read", **k)
    assert r(k=None) == NULL and r(k=tok(A, 128, -1)) == SHAPE and r(v=tok(B + 1)) == ALIGN
    assert r(k=tok(None), v=tok(None)) == OK  # nothing is wanted


def test_attention_rejects_bad_arguments(L):
    assert attend(L, q=None) == NULL and attend(L, o=None) == NULL and attend(L, q=tok(None)) == NULL
    assert attend(L, o=tok(None)) == NULL
    assert attend(L, Hq=3) == SHAPE and attend(L, Hq=0) == SHAPE and attend(L, q=tok(A, -1)) == SHAPE
    assert attend(L, q=tok(A + 1)) == ALIGN and attend(L, o=tok(C + 1)) == ALIGN and attend(L, lse=D + 2) == ALIGN
    for bad in (dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(window=2 ** 31), dict(sinks=4),
                dict(window=4, causal=0), dict(window=4, sinks=-1), dict(window=4, sinks=2 ** 31)):
        assert attend(L, **bad) == FLAGS, bad
    w = L.nvfp4_cache_attention_workspace
    assert w(-1, 4, 2, 64, 3) == SHAPE and w(4, 3, 2, 64, 3) == SHAPE and w(4, 4, 2, 48, 3) == SHAPE
    assert w(0, 4, 2, 64, 3) == 0 and w(4, 4, 2, 64, 0) == 0 and w(4, 4, 2, 64, 3) >= 0
    n = w(4, 4, 2, 64, 3)
    if n > 0:
        assert attend(L, ws=None) == NULL and attend(L, wn=n - 1) == SHAPE and attend(L, ws=A + 8) == ALIGN


def test_launch_failure_is_reported(L):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU: the fake device addresses would be launched")
    assert rope(L) == CUDA and grad(L) == CUDA and write(L) == CUDA and write(L, "nvfp4_cache_read") == CUDA
    assert attend(L) == CUDA


def test_binding_rejects_host_tensors():
    c = nv.nvfp4_kv_cache(2, 1, 16, 32, device="cpu")
    x = torch.zeros((1, 1, 32), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    calls = (lambda: nv.nvfp4_qk_rope(x, x, i[:1], torch.ones(16)),
             lambda: nv.nvfp4_qk_rope_backward(x, x, x, x, i[:1], torch.ones(16)),
             lambda: nv.nvfp4_cache_write(x, x, c, i, i[:1], i[:1, None]),
             lambda: nv.nvfp4_cache_read(c, i, i[:1], i[:1, None], tokens=1),
             lambda: nv.nvfp4_cache_attention(x, c, i, i[:1], i[:1, None]))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_binding_raises_without_the_library(monkeypatch, tmp_path):
    monkeypatch.setattr(attention, "_lib", None)
    monkeypatch.setattr(attention, "_LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="not built"):
        nv.attention_lib()
