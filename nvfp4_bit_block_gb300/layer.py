"""Python binding of the operators around the NVFP4 linear layer
(include/nvfp4_layer.h): argument checks and marshalling only; the work runs in
``_build/libnvfp4_layer.so``.  There is no CPU fallback.

* :func:`nvfp4_layernorm`, :func:`nvfp4_layernorm_backward`
* :func:`nvfp4_linear` -- NVFP4 operands, bias + activation + residual
* :func:`nvfp4_act_backward` -- gradient of the activation and the bias

Results are allocated on the stream that the call runs on (``stream``, or
torch's current one), as are workspaces, so torch's allocator hands their memory
out again in that stream's order.  To use a result on another stream, make that
stream wait and call ``record_stream`` on the tensor, as for any torch tensor.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

from .build import LAYER_LIB as _LIB_PATH

__all__ = ["ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_GELU_TANH", "ACT_SILU", "Normed", "NormGrads", "LinearOut",
           "ActGrads", "layer_lib", "nvfp4_layernorm", "nvfp4_layernorm_backward", "nvfp4_linear",
           "nvfp4_act_backward"]

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)

_lib: Optional[ctypes.CDLL] = None


def layer_lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"NVFP4 CUDA library not built ({_LIB_PATH}); call "
                               "nvfp4_bit_block_gb300.build() first")
        L = ctypes.CDLL(_LIB_PATH)
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sigs = {
            "nvfp4_layernorm": [p, i64, i64, i64, i32, p, p, i32, f32, p, i64, i32, p, p, p, p],
            "nvfp4_layernorm_backward": [p, i64, i32, p, i64, i32, i64, i64, p, p, p, i32, p, i64, p, i64, p, p, p, i64,
                                         p],
            "nvfp4_linear": [p, p, p, p, p, p, i64, i64, i64, p, i32, i32, p, i64, p, i64, p, i64, i32, p, p, i64, p, p],
            "nvfp4_act_backward": [p, i64, p, i64, i64, i64, i32, i32, p, i64, p, p, i64, p],
        }
        for name, args in sigs.items():
            f = getattr(L, name)
            f.restype, f.argtypes = i32, args
        for name, n in (("nvfp4_layernorm_backward_workspace", 2), ("nvfp4_linear_workspace", 3),
                        ("nvfp4_act_backward_workspace", 2)):
            f = getattr(L, name)
            f.restype, f.argtypes = i64, [i64] * n
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status < 0:
        from . import Nvfp4Error
        raise Nvfp4Error(status, where)


def _entered(stream):
    """Context in which `stream` (a torch stream or a raw cudaStream_t) is torch's current one."""
    import torch
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _is_bf16(t, name: str) -> int:
    """1 for bfloat16, 0 for float32."""
    import torch
    if t.dtype is torch.bfloat16:
        return 1
    if t.dtype is torch.float32:
        return 0
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float32 (got {t.dtype})")


def _matrix(t, name: str, device, shape=None, dtype=None):
    """(data_ptr, row stride) of a 2-D tensor on `device` with unit column stride."""
    if t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device} (got {t.device})")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must have shape {shape} (got {(rows, cols)})")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along columns")
    return t.data_ptr(), (t.stride(0) if rows > 1 else max(cols, 1))


def _vector(t, name: str, n: int, device, dtype=None):
    """data_ptr of a contiguous tensor of n elements on `device`, None for None."""
    if t is None:
        return None
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device} (got {t.device})")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements (got {tuple(t.shape)})")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    return t.data_ptr()


def _weights(gamma, beta, n: int, device):
    """(gamma pointer, beta pointer, is_bf16) of the norm's optional weights, both of one type."""
    bf16 = 0
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            bf16 = _is_bf16(t, name)
    if gamma is not None and beta is not None and gamma.dtype is not beta.dtype:
        raise TypeError("gamma and beta must have the same type")
    return _vector(gamma, "gamma", n, device), _vector(beta, "beta", n, device), bf16


def _call(name: str, device, args) -> None:
    """The C call on `device`'s current stream (appended to `args`)."""
    import torch
    fn = getattr(layer_lib(), name)
    index = device.index
    if index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    _check(st, name)


def _workspace(name: str, device, *sizes):
    """(tensor kept alive by the caller, pointer, bytes) of a call's scratch memory."""
    import torch
    fn = getattr(layer_lib(), name)
    if device.index == torch.cuda.current_device():
        n = fn(*sizes)
    else:
        with torch.cuda.device(device):
            n = fn(*sizes)
    _check(n, name)
    if n == 0:
        return None, None, 0
    t = torch.empty(n, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), n


@dataclass
class Normed:
    y: object
    mean: object  # float32[M], None if not asked for
    rstd: object  # float32[M], None if not asked for
    amax: object  # float32[2] for nvfp4_quantize, None if not asked for


@dataclass
class NormGrads:
    dx: object
    dgamma: object  # float32[N], None if not asked for
    dbeta: object   # float32[N], None if not asked for


@dataclass
class LinearOut:
    d: object
    z: object     # the activation's input, None if not asked for
    amax: object  # float32[2] for nvfp4_quantize, None if not asked for


@dataclass
class ActGrads:
    dz: object
    dbias: object  # float32[N], None if not asked for


def nvfp4_layernorm(x, gamma=None, beta=None, eps: float = 1e-5, out=None, out_dtype=None, want_stats: bool = True,
                    want_amax: bool = False, stream=None) -> Normed:
    """Layer norm of each row of x (M x N, bf16 or fp32): y of `out_dtype`
    (default: x's), the rows' mean and rstd for the backward pass, and with
    `want_amax` the amax that :func:`nvfp4_quantize` takes.  `out` may be x."""
    import torch
    if stream is not None:
        with _entered(stream):
            return nvfp4_layernorm(x, gamma, beta, eps, out, out_dtype, want_stats, want_amax)
    dev = x.device
    xp, ldx = _matrix(x, "x", dev)
    xb = _is_bf16(x, "x")
    M, N = x.shape
    gp, bp, wb = _weights(gamma, beta, N, dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or x.dtype, device=dev)
    yp, ldy = _matrix(out, "out", dev, (M, N), out_dtype)
    yb = _is_bf16(out, "out")
    mean = rstd = amax = None
    if want_stats:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
        rstd = torch.empty(M, dtype=torch.float32, device=dev)
    if want_amax:
        amax = torch.empty(2, dtype=torch.float32, device=dev)
    _call("nvfp4_layernorm", dev, (xp, M, N, ldx, xb, gp, bp, wb, eps, yp, ldy, yb,
                                   mean.data_ptr() if want_stats else None, rstd.data_ptr() if want_stats else None,
                                   amax.data_ptr() if want_amax else None))
    return Normed(out, mean, rstd, amax)


def nvfp4_layernorm_backward(dy, x, mean, rstd, gamma=None, dres=None, out=None, want_dgamma: bool = True,
                             want_dbeta: bool = True, stream=None) -> NormGrads:
    """Gradients of :func:`nvfp4_layernorm` from its input, mean and rstd: dx of
    x's type (plus `dres`, the residual branch's gradient) and the fp32 sums
    dgamma and dbeta.  `out` (dx) may be dy or dres."""
    import torch
    if stream is not None:
        with _entered(stream):
            return nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, dres, out, want_dgamma, want_dbeta)
    dev = x.device
    xp, ldx = _matrix(x, "x", dev)
    xb = _is_bf16(x, "x")
    M, N = x.shape
    dyp, lddy = _matrix(dy, "dy", dev, (M, N))
    dyb = _is_bf16(dy, "dy")
    rp, ldr = (None, 0) if dres is None else _matrix(dres, "dres", dev, (M, N), x.dtype)
    mp = _vector(mean, "mean", M, dev, torch.float32)
    sp = _vector(rstd, "rstd", M, dev, torch.float32)
    gp, _, wb = _weights(gamma, None, N, dev)
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=dev)
    op, ldo = _matrix(out, "out", dev, (M, N), x.dtype)
    dgamma = torch.empty(N, dtype=torch.float32, device=dev) if want_dgamma else None
    dbeta = torch.empty(N, dtype=torch.float32, device=dev) if want_dbeta else None
    ws, wp, wn = _workspace("nvfp4_layernorm_backward_workspace", dev, M, N) if want_dgamma or want_dbeta \
        else (None, None, 0)
    _call("nvfp4_layernorm_backward", dev,
          (dyp, lddy, dyb, xp, ldx, xb, M, N, mp, sp, gp, wb, rp, ldr, op, ldo,
           dgamma.data_ptr() if want_dgamma else None, dbeta.data_ptr() if want_dbeta else None, wp, wn))
    return NormGrads(out, dgamma, dbeta)


def nvfp4_linear(qa, sfa, alpha_a, qb, sfb, alpha_b, bias=None, act: int = ACT_NONE, residual=None, out=None,
                 out_dtype=None, want_z: bool = False, want_amax: bool = False, status=None, stream=None) -> LinearOut:
    """d = act(alpha_a * alpha_b * A * B^T + bias) + residual, bf16 (default) or
    fp32: qa (M x K/2: tokens) and qb (N x K/2: the weight's rows) are codes with
    K contiguous, sfa / sfb their scales in the tiled layout (SF_SWIZZLED),
    alpha_a / alpha_b one-element device views of the copies' alpha.  With
    `want_z` the activation's input is kept for :func:`nvfp4_act_backward`, with
    `want_amax` the amax that :func:`nvfp4_quantize` takes.  `residual` has d's
    type and may be `out`."""
    import torch
    if stream is not None:
        with _entered(stream):
            return nvfp4_linear(qa, sfa, alpha_a, qb, sfb, alpha_b, bias, act, residual, out, out_dtype, want_z,
                                want_amax, status)
    dev = qa.device
    M, half = qa.shape
    N, K = qb.shape[0], 2 * half
    if qb.shape[1] != half:
        raise ValueError("A and B must have the same K")
    u8, f32 = torch.uint8, torch.float32
    tiles = -(-(K // 16) // 4) * 4
    ap = _vector(qa, "qa", M * half, dev, u8)
    bp = _vector(qb, "qb", N * half, dev, u8)
    sap = _vector(sfa, "sfa", -(-M // 128) * 128 * tiles, dev, u8)
    sbp = _vector(sfb, "sfb", -(-N // 128) * 128 * tiles, dev, u8)
    aap = _vector(alpha_a, "alpha_a", 1, dev, f32)
    abp = _vector(alpha_b, "alpha_b", 1, dev, f32)
    biasp, biasb = (None, 0) if bias is None else (_vector(bias, "bias", N, dev), _is_bf16(bias, "bias"))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=dev)
    dp, ldd = _matrix(out, "out", dev, (M, N), out_dtype)
    ob = _is_bf16(out, "out")
    rp, ldr = (None, 0) if residual is None else _matrix(residual, "residual", dev, (M, N), out.dtype)
    z = amax = zp = amp = None
    if want_z:
        z = torch.empty((M, N), dtype=out.dtype, device=dev)
        zp = z.data_ptr()
    if want_amax:
        if not ob:
            raise TypeError("want_amax goes with a bfloat16 result (what nvfp4_quantize takes)")
        amax = torch.empty(2, dtype=f32, device=dev)
        amp = amax.data_ptr()
    ws, wp, wn = _workspace("nvfp4_linear_workspace", dev, M, N, K)
    _call("nvfp4_linear", dev, (ap, sap, aap, bp, sbp, abp, M, N, K, biasp, biasb, act, rp, ldr, zp, N, dp, ldd, ob,
                                amp, wp, wn, _vector(status, "status", 1, dev, torch.int32)))
    return LinearOut(out, z, amax)


def nvfp4_act_backward(dy, z, act: int, out=None, want_dz: bool = True, want_dbias: bool = True,
                       stream=None) -> ActGrads:
    """dz = dy * act'(z) (dy, z and dz of one type, bf16 or fp32) and the fp32
    bias gradient, the column sums of dz.  z may be None with ACT_NONE, where
    `want_dz=False` leaves the bias gradient alone.  `out` may be dy or z."""
    import torch
    if stream is not None:
        with _entered(stream):
            return nvfp4_act_backward(dy, z, act, out, want_dz, want_dbias)
    dev = dy.device
    dyp, lddy = _matrix(dy, "dy", dev)
    b = _is_bf16(dy, "dy")
    M, N = dy.shape
    zp, ldz = (None, 0) if z is None else _matrix(z, "z", dev, (M, N), dy.dtype)
    op, ldo = None, 0
    if want_dz:
        if out is None:
            out = torch.empty((M, N), dtype=dy.dtype, device=dev)
        op, ldo = _matrix(out, "out", dev, (M, N), dy.dtype)
    dbias = torch.empty(N, dtype=torch.float32, device=dev) if want_dbias else None
    ws, wp, wn = _workspace("nvfp4_act_backward_workspace", dev, M, N) if want_dbias else (None, None, 0)
    _call("nvfp4_act_backward", dev, (dyp, lddy, zp, ldz, M, N, b, act, op, ldo,
                                      dbias.data_ptr() if want_dbias else None, wp, wn))
    return ActGrads(out if want_dz else None, dbias)
