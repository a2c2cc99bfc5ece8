"""Python interface of the operators around the NVFP4 linear layer
(include/nvfp4_layer.h).  The work runs in ``_build/libnvfp4_layer.so``; argument
checks and result tensors are made by the extension ``_build/_nvfp4_layer.so``
(csrc/layer_binding.cpp).  There is no CPU fallback.

* :func:`nvfp4_layernorm`, :func:`nvfp4_layernorm_backward`
* :func:`nvfp4_linear` -- NVFP4 operands, bias + activation + residual
* :func:`nvfp4_act_backward` -- gradient of the activation and the bias

Matrices are 2-D CUDA tensors of bfloat16 or float32 with unit column stride;
wrong types raise TypeError, wrong shapes, strides or devices ValueError, and
what the library refuses Nvfp4Error.

Results are allocated on the stream that the call runs on (``stream``, a torch
stream or a raw cudaStream_t of the tensors' device, or torch's current one), as are workspaces, so
torch's allocator hands their memory out again in that stream's order.  To use a
result on another stream, make that stream wait and call ``record_stream`` on the
tensor, as for any torch tensor.  The small fp32 results of one call (mean, rstd
and amax; dgamma and dbeta) share one allocation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

from .build import LAYER_EXT as _EXT_PATH
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


_ext = None


def _binding():
    """The loaded extension.  Raises if it has not been built."""
    global _ext
    if _ext is None:
        import importlib.machinery
        import importlib.util
        layer_lib()
        if not os.path.exists(_EXT_PATH):
            raise RuntimeError(f"NVFP4 binding not built ({_EXT_PATH}); call nvfp4_bit_block_gb300.build() first")
        import torch  # noqa: F401  (the extension links its libraries)
        loader = importlib.machinery.ExtensionFileLoader("_nvfp4_layer", _EXT_PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_nvfp4_layer", loader))
        loader.exec_module(ext)
        _ext = ext
    return _ext


def _entered(stream, x):
    """Context in which `stream` (a torch stream or a raw cudaStream_t) is the current one of the device of x, the tensor
    that the call is on.  The raw handle 0 is the default stream (an ExternalStream of it would be a new stream of torch's
    pool)."""
    import torch
    if not getattr(x, "is_cuda", False):
        return contextlib.nullcontext()  # the call refuses it
    if not hasattr(stream, "cuda_stream"):  # a handle has no device of its own: it is taken for one of x's
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=x.device) if handle else torch.cuda.default_stream(x.device)
    elif stream.device != x.device:
        raise ValueError(f"stream must be on {x.device} (got {stream.device})")
    return torch.cuda.stream(stream)


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
    (default: out's or x's), the rows' mean and rstd for the backward pass, and
    with `want_amax` the amax that :func:`nvfp4_quantize` takes.  gamma and beta
    are bf16 or fp32 vectors of one type.  `out` may be x.  Rows of no values have
    mean and rstd NaN."""
    if stream is not None:
        with _entered(stream, x):
            return nvfp4_layernorm(x, gamma, beta, eps, out, out_dtype, want_stats, want_amax)
    return Normed(*(_ext or _binding()).layernorm(x, gamma, beta, eps, out, out_dtype, want_stats, want_amax))


def nvfp4_layernorm_backward(dy, x, mean, rstd, gamma=None, dres=None, out=None, want_dgamma: bool = True,
                             want_dbeta: bool = True, stream=None) -> NormGrads:
    """Gradients of :func:`nvfp4_layernorm` from its input, mean and rstd: dx of
    x's type (plus `dres`, the residual branch's gradient) and the fp32 sums
    dgamma and dbeta.  `out` (dx) may be dy or dres."""
    if stream is not None:
        with _entered(stream, x):
            return nvfp4_layernorm_backward(dy, x, mean, rstd, gamma, dres, out, want_dgamma, want_dbeta)
    return NormGrads(*(_ext or _binding()).layernorm_backward(dy, x, mean, rstd, gamma, dres, out, want_dgamma,
                                                              want_dbeta))


def nvfp4_linear(qa, sfa, alpha_a, qb, sfb, alpha_b, bias=None, act: int = ACT_NONE, residual=None, out=None,
                 out_dtype=None, want_z: bool = False, want_amax: bool = False, status=None, stream=None) -> LinearOut:
    """d = act(alpha_a * alpha_b * A * B^T + bias) + residual, bf16 (default) or
    fp32: qa (M x K/2: tokens) and qb (N x K/2: the weight's rows) are codes with
    K contiguous, sfa / sfb their scales in the tiled layout (SF_SWIZZLED),
    alpha_a / alpha_b one-element device views of the copies' alpha.  With
    `want_z` the activation's input is kept for :func:`nvfp4_act_backward`, with
    `want_amax` the amax that :func:`nvfp4_quantize` takes.  `residual` has d's
    type and may be `out`.  `status`: int32[1] on the device, as nvfp4_gemm's."""
    if stream is not None:
        with _entered(stream, qa):
            return nvfp4_linear(qa, sfa, alpha_a, qb, sfb, alpha_b, bias, act, residual, out, out_dtype, want_z,
                                want_amax, status)
    return LinearOut(*(_ext or _binding()).linear(qa, sfa, alpha_a, qb, sfb, alpha_b, bias, act, residual, out,
                                                  out_dtype, want_z, want_amax, status))


def nvfp4_act_backward(dy, z, act: int, out=None, want_dz: bool = True, want_dbias: bool = True,
                       stream=None) -> ActGrads:
    """dz = dy * act'(z) (dy, z and dz of one type, bf16 or fp32) and the fp32
    bias gradient, the column sums of dz.  z may be None with ACT_NONE, where
    `want_dz=False` leaves the bias gradient alone.  `out` may be dy or z."""
    if stream is not None:
        with _entered(stream, dy):
            return nvfp4_act_backward(dy, z, act, out, want_dz, want_dbias)
    return ActGrads(*(_ext or _binding()).act_backward(dy, z, act, out, want_dz, want_dbias))
