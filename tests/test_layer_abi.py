"""The C ABI of the operators around the linear layer (include/nvfp4_layer.h):
the library exports what the header declares and rejects bad arguments on the
host (no GPU needed: these calls return before any CUDA work is enqueued)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300 import layer
from nvfp4_bit_block_gb300.build import LAYER_LIB

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000  # fake aligned device addresses: never dereferenced
OK, NULL, SHAPE, ALIGN, FLAGS, CUDA = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def L():
    nv.build()
    return nv.layer_lib()


def test_library_exports_exactly_the_declared_entry_points(L):
    with open(os.path.join(ROOT, "include", "nvfp4_layer.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = sorted(re.findall(r"NVFP4_API\s+(?:int|int64_t)\s+(nvfp4_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", LAYER_LIB], capture_output=True, text=True).stdout
    assert sorted(set(re.findall(r"\bT (nvfp4_\w+)", out))) == declared
    assert {"nvfp4_layernorm", "nvfp4_layernorm_backward", "nvfp4_linear", "nvfp4_act_backward"} <= set(declared)
    for name in ("nvfp4_layernorm", "nvfp4_layernorm_backward", "nvfp4_linear", "nvfp4_act_backward"):
        assert callable(getattr(nv, name))


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "nvfp4_layer.h"\nint main(void) { return NVFP4_ACT_NONE; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def norm(L, **k):
    a = dict(x=A, M=4, N=32, ldx=32, xb=1, g=B, b=B, wb=0, eps=1e-5, y=C, ldy=32, yb=1, mean=D, rstd=D, amax=None)
    a.update(k)
    return L.nvfp4_layernorm(*a.values(), None)


def test_layernorm_rejects_bad_arguments(L):
    assert norm(L, M=-1) == SHAPE and norm(L, N=-1) == SHAPE and norm(L, M=2 ** 31) == SHAPE
    assert norm(L, ldx=31) == SHAPE and norm(L, ldy=31) == SHAPE and norm(L, ldx=2 ** 62) == SHAPE
    assert norm(L, eps=-1e-5) == FLAGS and norm(L, eps=float("nan")) == FLAGS and norm(L, eps=float("inf")) == FLAGS
    assert norm(L, x=None) == NULL and norm(L, y=None) == NULL
    assert norm(L, x=A + 1) == ALIGN and norm(L, y=C + 1) == ALIGN and norm(L, xb=0, x=A + 2) == ALIGN
    assert norm(L, g=B + 2) == ALIGN and norm(L, b=B + 1, wb=1) == ALIGN
    assert norm(L, mean=D + 2) == ALIGN and norm(L, rstd=D + 2) == ALIGN and norm(L, amax=D + 1) == ALIGN
    assert norm(L, M=0, x=None, y=None) == OK and norm(L, N=0, x=None, y=None) == OK  # nothing to do


def grad(L, **k):
    a = dict(dy=A, lddy=32, dyb=1, x=B, ldx=32, xb=1, M=4, N=32, mean=D, rstd=D, g=B, wb=0, dres=None, lddres=0, dx=C,
             lddx=32, dg=D, db=D, ws=A, wn=1 << 40)
    a.update(k)
    return L.nvfp4_layernorm_backward(*a.values(), None)


def test_layernorm_backward_rejects_bad_arguments(L):
    assert grad(L, M=-1) == SHAPE and grad(L, N=2 ** 31) == SHAPE
    assert grad(L, lddy=31) == SHAPE and grad(L, ldx=31) == SHAPE and grad(L, lddx=31) == SHAPE
    assert grad(L, dres=A, lddres=31) == SHAPE
    for p in ("dy", "x", "mean", "rstd", "dx"):
        assert grad(L, **{p: None}) == NULL, p
    assert grad(L, dy=A + 1) == ALIGN and grad(L, x=B + 1) == ALIGN and grad(L, dx=C + 1) == ALIGN
    assert grad(L, dres=A + 1, lddres=32) == ALIGN and grad(L, g=B + 2) == ALIGN
    assert grad(L, dg=D + 2) == ALIGN and grad(L, db=D + 2) == ALIGN
    assert L.nvfp4_layernorm_backward_workspace(-1, 4) == SHAPE
    assert L.nvfp4_layernorm_backward_workspace(0, 4) == 0 and L.nvfp4_layernorm_backward_workspace(4, 0) == 0
    assert grad(L, M=4, N=0, lddy=0, dg=None, db=None) == OK


def linear(L, **k):
    a = dict(qa=A, sfa=A, aa=D, qb=B, sfb=B, ab=D, M=4, N=40, K=64, bias=D, bb=0, act=0, res=None, ldr=0, z=None,
             ldz=0, d=C, ldd=40, ob=1, amax=None, ws=A, wn=1 << 40, status=None)
    a.update(k)
    return L.nvfp4_linear(*a.values(), None)


def test_linear_rejects_bad_arguments(L):
    assert linear(L, M=-1) == SHAPE and linear(L, N=-1) == SHAPE
    assert linear(L, K=0) == SHAPE and linear(L, K=48) == SHAPE and linear(L, K=-32) == SHAPE
    assert linear(L, ldd=39) == SHAPE and linear(L, res=A, ldr=39) == SHAPE and linear(L, z=A, ldz=39) == SHAPE
    assert linear(L, act=5) == FLAGS and linear(L, act=-1) == FLAGS
    for p in ("qa", "sfa", "aa", "qb", "sfb", "ab", "d"):
        assert linear(L, **{p: None}) == NULL, p
    assert linear(L, qa=A + 8) == ALIGN and linear(L, qb=B + 8) == ALIGN
    assert linear(L, sfa=A + 4) == ALIGN and linear(L, sfb=B + 4) == ALIGN
    assert linear(L, aa=D + 2) == ALIGN and linear(L, bias=D + 2) == ALIGN and linear(L, bias=D + 1, bb=1) == ALIGN
    assert linear(L, d=C + 1) == ALIGN and linear(L, d=C + 2, ob=0) == ALIGN
    assert linear(L, res=A + 1, ldr=40) == ALIGN and linear(L, z=A + 1, ldz=40) == ALIGN
    assert linear(L, amax=D + 2) == ALIGN and linear(L, status=D + 1) == ALIGN
    assert linear(L, M=0) == OK and linear(L, N=0) == OK
    assert L.nvfp4_linear_workspace(4, 4, 48) == SHAPE and L.nvfp4_linear_workspace(0, 4, 64) == 0


def act(L, **k):
    a = dict(dy=A, lddy=32, z=B, ldz=32, M=4, N=32, b=1, act=1, dz=C, lddz=32, db=D, ws=A, wn=1 << 40)
    a.update(k)
    return L.nvfp4_act_backward(*a.values(), None)


def test_act_backward_rejects_bad_arguments(L):
    assert act(L, M=-1) == SHAPE and act(L, N=-1) == SHAPE
    assert act(L, lddy=31) == SHAPE and act(L, ldz=31) == SHAPE and act(L, lddz=31) == SHAPE
    assert act(L, act=5) == FLAGS and act(L, act=-1) == FLAGS
    assert act(L, dy=None) == NULL and act(L, z=None) == NULL
    assert act(L, dy=A + 1) == ALIGN and act(L, z=B + 1) == ALIGN and act(L, dz=C + 1) == ALIGN
    assert act(L, db=D + 2) == ALIGN and act(L, b=0, dy=A + 2) == ALIGN
    assert act(L, dz=None, db=None) == OK  # nothing asked for
    assert L.nvfp4_act_backward_workspace(4, -1) == SHAPE and L.nvfp4_act_backward_workspace(0, 4) == 0


def test_workspaces_are_checked(L):
    """Where a call needs scratch memory, NULL and a short buffer are refused."""
    n = L.nvfp4_layernorm_backward_workspace(16384, 5120)
    assert n >= 0
    if n > 0:
        big = dict(M=16384, N=5120, lddy=5120, ldx=5120, lddx=5120)
        assert grad(L, **big, ws=None) == NULL and grad(L, **big, wn=n - 1) == SHAPE
        assert grad(L, **big, ws=A + 4) == ALIGN
    n = L.nvfp4_act_backward_workspace(16384, 5120)
    assert n >= 0
    if n > 0:
        big = dict(M=16384, N=5120, lddy=5120, ldz=5120, lddz=5120)
        assert act(L, **big, ws=None) == NULL and act(L, **big, wn=n - 1) == SHAPE and act(L, **big, ws=A + 4) == ALIGN
    n = L.nvfp4_linear_workspace(1, 5120, 20480)
    assert n >= 0
    if n > 0:
        tall = dict(M=1, N=5120, K=20480, ldd=5120)
        assert linear(L, **tall, ws=None) == NULL and linear(L, **tall, wn=n - 1) == SHAPE


def test_launch_failure_is_reported(L):
    """Without a GPU, calls that pass the host checks fail in the CUDA runtime
    before anything runs, and say so."""
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU: the fake device addresses would be launched")
    assert norm(L) == CUDA and grad(L) == CUDA and linear(L) == CUDA and act(L) == CUDA


def test_binding_rejects_host_tensors_and_wrong_types():
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        nv.nvfp4_layernorm(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        nv.nvfp4_layernorm_backward(x, x, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        nv.nvfp4_act_backward(x, x, nv.ACT_GELU)
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((128, 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        nv.nvfp4_linear(q, s, torch.ones(1), q, s, torch.ones(1))
    with pytest.raises(ValueError, match="same K"):
        nv.nvfp4_linear(q, s, torch.ones(1), q[:, :16], s, torch.ones(1))
    with pytest.raises(TypeError):
        nv.nvfp4_layernorm(torch.zeros(4, dtype=torch.bfloat16))


def test_binding_raises_without_the_library(monkeypatch, tmp_path):
    monkeypatch.setattr(layer, "_lib", None)
    monkeypatch.setattr(layer, "_LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="not built"):
        nv.layer_lib()


def test_argument_counts_match_the_header(L):
    """The binding's signatures have the header's number of arguments."""
    with open(os.path.join(ROOT, "include", "nvfp4_layer.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for name, args in re.findall(r"NVFP4_API\s+\w+\s+(nvfp4_\w+)\s*\((.*?)\)\s*;", text, flags=re.S):
        f = getattr(L, name)
        assert len(f.argtypes) == args.count(",") + 1, name
        kinds = [ctypes.c_void_p if "*" in x else {"int64_t": ctypes.c_int64, "int": ctypes.c_int,
                                                   "float": ctypes.c_float}[x.split()[0]] for x in args.split(",")]
        assert list(f.argtypes) == kinds, name
