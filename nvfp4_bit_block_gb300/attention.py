"""Python interface of the attention operators on an NVFP4 cache
(include/nvfp4_attention.h).  The work runs in ``_build/libnvfp4_attention.so``;
argument checks and result tensors are made by the extension
``_build/_nvfp4_attention.so`` (csrc/attention_binding.cpp).  There is no CPU fallback.

* :func:`nvfp4_qk_rope`, :func:`nvfp4_qk_rope_backward` -- norm and rotation of queries
  and keys
* :func:`nvfp4_kv_cache` -- a paged cache of keys and values in 4 bits
* :func:`nvfp4_cache_write`, :func:`nvfp4_cache_read`
* :func:`nvfp4_cache_attention` -- prompts and single tokens, sliding window and sinks

Token tensors are 3-D CUDA tensors (tokens, heads, values) with contiguous values and any
stride from token to token and from head to head; wrong types raise TypeError, wrong
shapes, strides or devices ValueError, and what the library refuses Nvfp4Error.

A batch is three int32 tensors.  Sequence b holds ``lengths[b]`` tokens in the cache, on the
pages that row b of ``pages`` names in order; the call's rows ``starts[b]`` ..
``starts[b + 1] - 1`` are its last tokens.  Numbers out of range set ``status`` (int32[1])
to NVFP4_ERR_INDEX and are left out.

Results are allocated and streams are taken as in :mod:`.layer`.  Rows that belong to no
sequence (behind ``starts[-1]``, in a padded batch) are left as they are: in a result that
the call allocates they hold whatever its memory held, so pass ``out`` where they are used.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

from .build import ATTENTION_EXT as _EXT_PATH
from .build import ATTENTION_LIB as _LIB_PATH
from .layer import _entered

__all__ = ["KVCache", "QKRope", "QKRopeGrads", "CacheTokens", "AttentionOut", "attention_lib", "nvfp4_qk_rope",
           "nvfp4_qk_rope_backward", "nvfp4_kv_cache", "nvfp4_cache_write", "nvfp4_cache_read",
           "nvfp4_cache_attention"]

_lib: Optional[ctypes.CDLL] = None


class Tokens(ctypes.Structure):
    """nvfp4_tokens of the C ABI."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Cache(ctypes.Structure):
    """nvfp4_kv_cache of the C ABI."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "alpha_dev")]
                + [("pages", ctypes.c_int64)] + [(n, ctypes.c_int) for n in ("heads", "page_size", "dim")]
                + [(n, ctypes.c_int64) for n in ("code_page", "code_head", "code_row", "scale_page", "scale_head",
                                                 "scale_row")])


class Batch(ctypes.Structure):
    """nvfp4_batch of the C ABI."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("starts", "lengths", "table")]
                + [(n, ctypes.c_int64) for n in ("sequences", "table_width", "table_stride")])


def attention_lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"NVFP4 CUDA library not built ({_LIB_PATH}); call "
                               "nvfp4_bit_block_gb300.build() first")
        L = ctypes.CDLL(_LIB_PATH)
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sigs = {
            "nvfp4_qk_rope": [p, p, i32, i64, i32, i32, i32, i32, i32, p, p, i32, f32, p, p, i32, p, p, i32, p],
            "nvfp4_qk_rope_backward": [p, p, i32, p, p, i32, i64, i32, i32, i32, i32, i32, p, p, i32, f32, p, p, i32, p, p,
                                       p, p, p, i64, p],
            "nvfp4_cache_write": [p, p, i32, i64, p, p, p, p],
            "nvfp4_cache_read": [p, p, i32, i64, p, p, p, p],
            "nvfp4_cache_attention": [p, i64, i32, p, p, f32, i32, i64, i64, p, p, p, i64, p, p],
        }
        for name, args in sigs.items():
            f = getattr(L, name)
            f.restype, f.argtypes = i32, args
        for name, args in (("nvfp4_qk_rope_backward_workspace", [i64, i32, i32, i32]),
                           ("nvfp4_cache_attention_workspace", [i64, i32, i32, i32, i64])):
            f = getattr(L, name)
            f.restype, f.argtypes = i64, args
        _lib = L
    return _lib


_ext = None


def _binding():
    """The loaded extension.  Raises if it has not been built."""
    global _ext
    if _ext is None:
        import importlib.machinery
        import importlib.util
        attention_lib()
        if not os.path.exists(_EXT_PATH):
            raise RuntimeError(f"NVFP4 binding not built ({_EXT_PATH}); call nvfp4_bit_block_gb300.build() first")
        import torch  # noqa: F401  (the extension links its libraries)
        loader = importlib.machinery.ExtensionFileLoader("_nvfp4_attention", _EXT_PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_nvfp4_attention", loader))
        loader.exec_module(ext)
        _ext = ext
    return _ext


@dataclass
class KVCache:
    """A paged cache: codes uint8 (pages, heads, rows of a page, dim / 2), scales uint8
    (pages, heads, rows, dim / 16), keys and values with the same strides, in any order of
    pages, heads and rows; alpha float32[2], the tensor scales of keys and values."""
    k_codes: object
    k_scales: object
    v_codes: object
    v_scales: object
    alpha: object

    def tensors(self):
        return self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.alpha


@dataclass
class QKRope:
    q: object
    k: object


@dataclass
class QKRopeGrads:
    dq: object
    dk: object
    dgamma_q: object  # float32[D], None without the norm or if not asked for
    dgamma_k: object


@dataclass
class CacheTokens:
    k: object
    v: object


@dataclass
class AttentionOut:
    o: object
    lse: object  # float32 (tokens, heads), None if not asked for


def nvfp4_kv_cache(pages: int, heads: int, page_size: int, dim: int, alpha=(2.0 ** -5, 2.0 ** -5),
                   device="cuda") -> KVCache:
    """An empty cache of `pages` pages of `page_size` tokens (a multiple of 16), `dim` values a
    head (a multiple of 32, at most 256).  alpha: the tensor scales of keys and values, best
    powers of two: values up to 2688 alpha are held; blocks of 16 whose largest value is below
    0.094 alpha have scales of fewer bits, and at or below alpha / 171 they become zeros."""
    import torch
    new = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device)
    k, v = new(pages, heads, page_size, dim // 2), new(pages, heads, page_size, dim // 2)
    sk, sv = new(pages, heads, page_size, dim // 16), new(pages, heads, page_size, dim // 16)
    return KVCache(k, sk, v, sv, torch.tensor(alpha, dtype=torch.float32, device=device))


def nvfp4_qk_rope(q, k, positions, inv_freq, gamma_q=None, gamma_k=None, eps: float = 1e-6, norm: bool = True,
                  interleaved: bool = False, out_q=None, out_k=None, out_dtype=None, stream=None) -> QKRope:
    """Queries (T, Hq, D) and keys (T, Hk, D), bf16 or fp32, each head normalised by its root
    mean square (times gamma, bf16 or fp32 weights of one type) and turned: pair i of the first
    2 * len(inv_freq) values by positions[t] * inv_freq[i].  A pair is values (i, i + len), or
    with `interleaved` neighbours (2i, 2i + 1).  With norm=False only turned.  The results are of
    `out_dtype` (default: out's or q's); out_q and out_k may be q and k."""
    if stream is not None:
        with _entered(stream, q):
            return nvfp4_qk_rope(q, k, positions, inv_freq, gamma_q, gamma_k, eps, norm, interleaved, out_q, out_k,
                                 out_dtype)
    return QKRope(*(_ext or _binding()).qk_rope(q, k, positions, inv_freq, gamma_q, gamma_k, eps, norm, interleaved,
                                                out_q, out_k, out_dtype))


def nvfp4_qk_rope_backward(dq, dk, q, k, positions, inv_freq, gamma_q=None, gamma_k=None, eps: float = 1e-6,
                           norm: bool = True, interleaved: bool = False, out_q=None, out_k=None,
                           want_dgamma: bool = True, stream=None) -> QKRopeGrads:
    """Gradients of :func:`nvfp4_qk_rope` from those of its results and its inputs: dq and dk of
    q's type and the fp32 sums dgamma_q and dgamma_k.  With norm=False q and k are not read and
    may be None.  out_q and out_k may be dq and dk, or q and k."""
    if stream is not None:
        with _entered(stream, dq):
            return nvfp4_qk_rope_backward(dq, dk, q, k, positions, inv_freq, gamma_q, gamma_k, eps, norm, interleaved,
                                          out_q, out_k, want_dgamma)
    return QKRopeGrads(*(_ext or _binding()).qk_rope_backward(dq, dk, q, k, positions, inv_freq, gamma_q, gamma_k, eps,
                                                              norm, interleaved, out_q, out_k, want_dgamma))


def nvfp4_cache_write(k, v, cache: KVCache, starts, lengths, pages, status=None, stream=None) -> None:
    """Quantize the batch's keys and values (T, heads, dim; bf16 or fp32) into the cache.
    `lengths` count the new tokens.  NaN and infinities are stored as 0 and the largest code and
    set `status` to NVFP4_ERR_NONFINITE.  No two rows may lie in one place of the cache."""
    if stream is not None:
        with _entered(stream, k):
            return nvfp4_cache_write(k, v, cache, starts, lengths, pages, status)
    (_ext or _binding()).cache_write(k, v, *cache.tensors(), starts, lengths, pages, status)


def nvfp4_cache_read(cache: KVCache, starts, lengths, pages, tokens: Optional[int] = None, out_k=None, out_v=None,
                     out_dtype=None, want_k: bool = True, want_v: bool = True, status=None,
                     stream=None) -> CacheTokens:
    """The batch's keys and values out of the cache, (tokens, heads, dim) in bf16 (default) or
    fp32: the last starts[b + 1] - starts[b] tokens of each sequence.  `tokens` is the number of
    rows where no result is given (starts[-1] as the host knows it)."""
    if stream is not None:
        with _entered(stream, cache.k_codes):
            return nvfp4_cache_read(cache, starts, lengths, pages, tokens, out_k, out_v, out_dtype, want_k, want_v,
                                    status)
    return CacheTokens(*(_ext or _binding()).cache_read(*cache.tensors(), starts, lengths, pages, tokens, out_k, out_v,
                                                        out_dtype, want_k, want_v, status))


def nvfp4_cache_attention(q, cache: KVCache, starts, lengths, pages, scale: Optional[float] = None,
                          causal: bool = True, window: int = 0, sinks: int = 0, out=None, want_lse: bool = False,
                          status=None, stream=None) -> AttentionOut:
    """The batch's queries (T, Hq, dim; bf16) attend to the cache; Hq is a multiple of the
    cache's heads, and the tokens' own keys and values are in the cache already.  Key j is
    visible from position p if j <= p and, with window > 0, p - j < window or j < sinks;
    with causal=False all of a sequence's keys are.  scale: default dim ** -0.5.  A row that
    sees nothing becomes zeros, its lse -inf.  `out` may be q."""
    if stream is not None:
        with _entered(stream, q):
            return nvfp4_cache_attention(q, cache, starts, lengths, pages, scale, causal, window, sinks, out, want_lse,
                                         status)
    return AttentionOut(*(_ext or _binding()).cache_attention(q, *cache.tensors(), starts, lengths, pages, scale, causal,
                                                              window, sinks, out, want_lse, status))
