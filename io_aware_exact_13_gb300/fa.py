"""Python binding of the C ABI in ``include/fa.h`` (argument marshalling only).

Every function here forwards device pointers, sizes and the current CUDA
stream to ``libfa.so``; all arithmetic runs in the library's CUDA kernels.
There is no CPU fallback: importing this module fails loudly when the library
has not been built, and every call raises if the library returns an error.

Names follow the C ABI: ``fa_fwd`` (bf16), ``fa_fwd_fp16``, ``fa_fwd_fp32``,
``fa_fwd_masked`` / ``fa_fwd_masked_fp16`` (a shared mask packed in a workspace),
``fa_fwd_dropout`` / ``fa_fwd_dropout_fp16`` (dropout on the probabilities),
``fa_fwd_splitkv`` / ``fa_fwd_splitkv_fp16`` (decoding), ``fa_bwd`` /
``fa_bwd_fp16`` (backward by recomputation), ``fa_fwd_varlen`` /
``fa_fwd_varlen_fp16`` (packed variable-length batches), ``fa_fwd_kvq8`` /
``fa_fwd_kvq8_fp16`` (decoding over an 8-bit cache), ``fa_fwd_cross`` / ``fa_bwd_cross`` and their ``_fp16`` forms
(keys of another length), their sizing helpers,
``fa_status_string``, ``fa_get_device_status``, ``fa_num_sms``. ``attention``,
``attention_decode``, ``attention_varlen``, ``attention_kvq8``, ``attention_cross``,
``attention_cross_backward`` and ``attention_backward`` are convenience wrappers
that allocate outputs (and the workspaces) with torch and pick the entry point from the dtype; ``kvq8_append`` and
``kvq8_read`` write and read the 8-bit cache (``KVCacheQ8``, allocated by ``kv_cache_q8``).
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

import torch

# Private names of torch that save host time on the calls beside kernels of a few microseconds, where this torch has them
# (None: the public way is taken).
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -m io_aware_exact_13_gb300.build` "
        "(there is no fallback implementation)")
lib = ctypes.CDLL(_LIB_PATH)

FA_OK = 0
FA_ERR_NULL = -1
FA_ERR_ALIGN = -2
FA_ERR_SHAPE = -3
FA_ERR_UNSUPPORTED = -4
FA_ERR_LAUNCH = -5
FA_ERR_TIMEOUT = -6
FA_ERR_WORKSPACE = -7
FA_ERR_SEQLENS = -8
FA_ERR_ARG = -9
FA_ERR_PAGE = -10
FA_ERR_VALUE = -11

# Every symbol the header declares, with its ctypes signature.
_vp = ctypes.c_void_p
_FWD_ARGS = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
             ctypes.c_float, ctypes.c_int, _vp]
SIGNATURES = {
    "fa_fwd": (ctypes.c_int, _FWD_ARGS),
    "fa_fwd_fp16": (ctypes.c_int, _FWD_ARGS),
    "fa_fwd_fp32": (ctypes.c_int, _FWD_ARGS),
    "fa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fa_get_device_status": (ctypes.c_int, [_vp]),
    "fa_num_sms": (ctypes.c_int, []),
    "fa_fwd_bias": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 4 + [ctypes.c_float, ctypes.c_int, _vp]),
    "fa_fwd_bias_fp16": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 4 + [ctypes.c_float, ctypes.c_int, _vp]),
    "fa_fwd_gqa": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int, _vp]),
    "fa_fwd_masked_workspace_bytes": (ctypes.c_longlong, [ctypes.c_int] * 2),
    "fa_fwd_dropout": (ctypes.c_int, [_vp] * 5 + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int, ctypes.c_float,
                                                                       ctypes.c_ulonglong, ctypes.c_ulonglong, _vp]),
    "fa_fwd_dropout_fp16": (ctypes.c_int, [_vp] * 5 + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int,
                                                                            ctypes.c_float, ctypes.c_ulonglong,
                                                                            ctypes.c_ulonglong, _vp]),
    "fa_fwd_masked": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int, _vp,
                                                                        ctypes.c_ulonglong, _vp]),
    "fa_fwd_masked_fp16": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int, _vp,
                                                                             ctypes.c_ulonglong, _vp]),
    "fa_fwd_gqa_fp16": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int, _vp]),
    "fa_splitkv_num_splits": (ctypes.c_int, [ctypes.c_int] * 5),
    "fa_splitkv_workspace_bytes": (ctypes.c_longlong, [ctypes.c_int] * 5),
    "fa_fwd_splitkv": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp] + [ctypes.c_int] * 5 +
                       [ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_ulonglong, _vp]),
    "fa_fwd_splitkv_fp16": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp] + [ctypes.c_int] * 5 +
                            [ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_ulonglong, _vp]),
    "fa_fwd_splitkv_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp] + [ctypes.c_int] * 5 +
                               [ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp]),
    "fa_fwd_varlen": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 6 + [ctypes.c_float, ctypes.c_int, _vp]),
    "fa_fwd_varlen_fp16": (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 6 + [ctypes.c_float, ctypes.c_int, _vp]),
    "fa_bwd_cross_workspace_bytes": (ctypes.c_longlong, [ctypes.c_int] * 6),
    "fa_cross_num_splits": (ctypes.c_int, [ctypes.c_int] * 4),
    "fa_kvq8_num_parts": (ctypes.c_int, [ctypes.c_int] * 6),
    "fa_kvq8_workspace_bytes": (ctypes.c_longlong, [ctypes.c_int] * 5),
    "fa_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_ulonglong, _vp]),
    "fa_fwd_host": (ctypes.c_int, [_vp] * 10 + [ctypes.c_int] * 4 + [ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp]),
    "fa_fwd_host_fp16": (ctypes.c_int, [_vp] * 10 + [ctypes.c_int] * 4 +
                         [ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp]),
    "fa_bwd_workspace_bytes": (ctypes.c_longlong, [ctypes.c_int] * 4),
    "fa_bwd": (ctypes.c_int, [_vp] * 9 + [ctypes.c_int] * 4 + [ctypes.c_float, ctypes.c_int, _vp,
                                                                 ctypes.c_ulonglong, _vp]),
    "fa_bwd_fp16": (ctypes.c_int, [_vp] * 9 + [ctypes.c_int] * 4 + [ctypes.c_float, ctypes.c_int, _vp,
                                                                      ctypes.c_ulonglong, _vp]),
}
_KVQ8_APPEND = [_vp] * 2 + [ctypes.c_longlong] * 4 + [_vp] * 2 + [ctypes.c_int] * 3 + [_vp] * 5 + [ctypes.c_int] * 6 + [_vp]
_KVQ8_READ = [_vp] * 5 + [ctypes.c_int] * 3 + [_vp] * 2 + [ctypes.c_int] * 3 + [_vp] * 2 + [ctypes.c_int] * 3 + [_vp]
_KVQ8_FWD = ([_vp] * 6 + [ctypes.c_int] * 3 + [_vp] * 3 + [ctypes.c_int] * 7 + [ctypes.c_float] + [ctypes.c_int] * 2 +
             [_vp, ctypes.c_ulonglong, _vp])
for _suffix in ("", "_fp16"):
    SIGNATURES["fa_kvq8_append" + _suffix] = (ctypes.c_int, _KVQ8_APPEND)
    SIGNATURES["fa_kvq8_read" + _suffix] = (ctypes.c_int, _KVQ8_READ)
    SIGNATURES["fa_fwd_kvq8" + _suffix] = (ctypes.c_int, _KVQ8_FWD)
    SIGNATURES["fa_fwd_cross" + _suffix] = (ctypes.c_int, [_vp] * 6 + [ctypes.c_int] * 6 +
                                            [ctypes.c_float, ctypes.c_int, _vp, ctypes.c_ulonglong, _vp])
    SIGNATURES["fa_bwd_cross" + _suffix] = (ctypes.c_int, [_vp] * 10 + [ctypes.c_int] * 6 +
                                            [ctypes.c_float, _vp, ctypes.c_ulonglong, _vp])
for _name, (_res, _args) in SIGNATURES.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")
        self.status = status


def fa_status_string(status: int) -> str:
    return lib.fa_status_string(int(status)).decode()


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _raw_fwd(fn_name, q, k, v, mask, out, lse, B, H, N, d, scale, causal, stream):
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), _ptr(lse), int(B), int(H), int(N),
                               int(d), float(scale), int(bool(causal)), ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def _check(q, k, v, mask, out, lse, dtype):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape or out.shape != q.shape:
        raise ValueError("q, k, v, out must all be [B, H, N, d]")
    B, H, N, d = q.shape
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, N):
        raise ValueError("lse must be a contiguous CUDA float32 [B, H, N] tensor")
    if mask is not None and (mask.dtype != torch.float32 or not mask.is_cuda or not mask.is_contiguous()
                             or mask.shape != (B, N, N)):
        raise ValueError("mask must be a contiguous CUDA float32 [B, N, N] tensor")
    return B, H, N, d


def fa_fwd(q, k, v, mask_or_null, out, lse, scale, causal, stream=None):
    """bf16 forward into caller-provided ``out`` [B,H,N,d] and ``lse`` [B,H,N]."""
    B, H, N, d = _check(q, k, v, mask_or_null, out, lse, torch.bfloat16)
    _raw_fwd("fa_fwd", q, k, v, mask_or_null, out, lse, B, H, N, d, scale, causal, stream)


def fa_fwd_fp16(q, k, v, mask_or_null, out, lse, scale, causal, stream=None):
    """fp16 forward into caller-provided ``out`` and ``lse``."""
    B, H, N, d = _check(q, k, v, mask_or_null, out, lse, torch.float16)
    _raw_fwd("fa_fwd_fp16", q, k, v, mask_or_null, out, lse, B, H, N, d, scale, causal, stream)


def fa_fwd_fp32(q, k, v, mask_or_null, out, lse, scale, causal, stream=None):
    """fp32 forward (fp32 arithmetic on the CUDA cores) into caller-provided ``out`` and ``lse``."""
    B, H, N, d = _check(q, k, v, mask_or_null, out, lse, torch.float32)
    _raw_fwd("fa_fwd_fp32", q, k, v, mask_or_null, out, lse, B, H, N, d, scale, causal, stream)


_BY_DTYPE = {torch.bfloat16: fa_fwd, torch.float16: fa_fwd_fp16, torch.float32: fa_fwd_fp32}


def attention(q, k, v, mask=None, scale=None, causal=False, out=None, lse=None, stream=None):
    """O, lse = softmax(scale * q k^T + mask) v for [B,H,N,d] CUDA tensors. A bf16 / fp16
    forward with a mask goes through ``fa_fwd_masked`` with a workspace from torch."""
    if q.dtype not in _BY_DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if mask is not None and q.dtype in _MASKED:
        ws = torch.empty(fa_fwd_masked_workspace_bytes(B, N), dtype=torch.uint8, device=q.device)
        _MASKED[q.dtype](q, k, v, mask, out, lse, scale, causal, ws, stream)
    else:
        _BY_DTYPE[q.dtype](q, k, v, mask, out, lse, scale, causal, stream)
    return out, lse


# ---------------------------------------------------------------- additive mask, packed
def fa_fwd_masked_workspace_bytes(B, N) -> int:
    n = int(lib.fa_fwd_masked_workspace_bytes(int(B), int(N)))
    if n < 0:
        raise FAError(n, "fa_fwd_masked_workspace_bytes")
    return n


def _fwd_masked(fn_name, dtype, q, k, v, mask, out, lse, scale, causal, workspace, stream):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, N, d) or v.shape != k.shape or out.shape != q.shape or H % Hkv:
        raise ValueError("q, out: [B, H, N, d]; k, v: [B, Hkv, N, d] with Hkv dividing H")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, N):
        raise ValueError("lse must be a contiguous CUDA float32 [B, H, N] tensor")
    if (mask is None or mask.dtype != torch.float32 or mask.shape != (B, N, N) or not mask.is_contiguous()
            or not mask.is_cuda):
        raise ValueError("mask must be a contiguous CUDA float32 [B, N, N] tensor")
    if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), _ptr(lse), B, H, Hkv, N, d,
                               float(scale), int(bool(causal)), _ptr(workspace), nbytes,
                               ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_fwd_masked(q, k, v, mask, out, lse, scale, causal, workspace, stream=None):
    """bf16 forward with a shared [B, N, N] fp32 mask, packed to one bit per entry in ``workspace``
    (at least ``fa_fwd_masked_workspace_bytes(B, N)`` bytes) when its entries are all 0 or -inf;
    k, v may hold fewer heads (grouped-query)."""
    _fwd_masked("fa_fwd_masked", torch.bfloat16, q, k, v, mask, out, lse, scale, causal, workspace, stream)


def fa_fwd_masked_fp16(q, k, v, mask, out, lse, scale, causal, workspace, stream=None):
    """fp16 forward with a shared mask and a workspace (see ``fa_fwd_masked``)."""
    _fwd_masked("fa_fwd_masked_fp16", torch.float16, q, k, v, mask, out, lse, scale, causal, workspace, stream)


_MASKED = {torch.bfloat16: fa_fwd_masked, torch.float16: fa_fwd_masked_fp16}


# ---------------------------------------------------------------- dropout
def _fwd_dropout(fn_name, dtype, q, k, v, out, lse, scale, causal, p_drop, seed, offset, stream):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, N, d) or v.shape != k.shape or out.shape != q.shape or H % Hkv:
        raise ValueError("q, out: [B, H, N, d]; k, v: [B, Hkv, N, d] with Hkv dividing H")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, N):
        raise ValueError("lse must be a contiguous CUDA float32 [B, H, N] tensor")
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, N, d, float(scale),
                               int(bool(causal)), float(p_drop), int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                               ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_fwd_dropout(q, k, v, out, lse, scale, causal, p_drop, seed, offset=0, stream=None):
    """bf16 forward with dropout: keep decisions from Philox4x64-10 keyed by ``seed``, counter
    {query row, key / 32, b*H + h, ``offset``}; k, v may hold fewer heads (grouped-query)."""
    _fwd_dropout("fa_fwd_dropout", torch.bfloat16, q, k, v, out, lse, scale, causal, p_drop, seed, offset, stream)


def fa_fwd_dropout_fp16(q, k, v, out, lse, scale, causal, p_drop, seed, offset=0, stream=None):
    """fp16 forward with dropout (see ``fa_fwd_dropout``)."""
    _fwd_dropout("fa_fwd_dropout_fp16", torch.float16, q, k, v, out, lse, scale, causal, p_drop, seed, offset, stream)


def attention_dropout(q, k, v, p_drop, seed, offset=0, scale=None, causal=False, stream=None):
    """Forward with dropout; allocates O and lse."""
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fn = {torch.bfloat16: fa_fwd_dropout, torch.float16: fa_fwd_dropout_fp16}[q.dtype]
    fn(q, k, v, out, lse, scale, causal, p_drop, seed, offset, stream)
    return out, lse


# ---------------------------------------------------------------- forward from host memory
def fa_fwd_host(q_host, k_host, v_host, out_host, lse_host, q_dev, k_dev, v_dev, out_dev, lse_dev, scale, causal,
                n_chunks=4, stream=None):
    """Forward with inputs and outputs in (pinned) host tensors; the device tensors
    are caller-owned staging buffers. Copies and compute are pipelined over head
    chunks; synchronise the stream before reading out_host / lse_host."""
    dtype = q_host.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("bf16 or fp16 inputs")
    for name, t in (("q_host", q_host), ("k_host", k_host), ("v_host", v_host), ("out_host", out_host)):
        if t.dtype != dtype or t.is_cuda or not t.is_contiguous() or t.shape != q_host.shape:
            raise ValueError(f"{name} must be a contiguous host {dtype} tensor shaped like q_host")
    for name, t in (("q_dev", q_dev), ("k_dev", k_dev), ("v_dev", v_dev), ("out_dev", out_dev)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or t.shape != q_host.shape:
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor shaped like q_host")
    B, H, N, d = q_host.shape
    for name, t, cuda in (("lse_host", lse_host, False), ("lse_dev", lse_dev, True)):
        if t.dtype != torch.float32 or t.is_cuda != cuda or not t.is_contiguous() or t.shape != (B, H, N):
            raise ValueError(f"{name} must be a contiguous float32 [B, H, N] tensor")
    fn = lib.fa_fwd_host if dtype == torch.bfloat16 else lib.fa_fwd_host_fp16
    rc = fn(*[_ptr(t) for t in (q_host, k_host, v_host, out_host, lse_host, q_dev, k_dev, v_dev, out_dev, lse_dev)],
            B, H, N, d, float(scale), int(bool(causal)), int(n_chunks), ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_host")


# ---------------------------------------------------------------- grouped-query attention
def _fwd_gqa(fn_name, dtype, q, k, v, mask_or_null, out, lse, scale, causal, stream):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, N, d) or v.shape != k.shape or out.shape != q.shape or H % Hkv:
        raise ValueError("q, out: [B, H, N, d]; k, v: [B, Hkv, N, d] with Hkv dividing H")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, N):
        raise ValueError("lse must be a contiguous CUDA float32 [B, H, N] tensor")
    if mask_or_null is not None and (mask_or_null.dtype != torch.float32 or mask_or_null.shape != (B, N, N)
                                     or not mask_or_null.is_contiguous() or not mask_or_null.is_cuda):
        raise ValueError("mask must be a contiguous CUDA float32 [B, N, N] tensor")
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(mask_or_null), _ptr(out), _ptr(lse), B, H, Hkv, N, d,
                               float(scale), int(bool(causal)), ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_fwd_gqa(q, k, v, mask_or_null, out, lse, scale, causal, stream=None):
    """bf16 grouped-query forward: k, v are [B, Hkv, N, d], shared by H / Hkv query heads each."""
    _fwd_gqa("fa_fwd_gqa", torch.bfloat16, q, k, v, mask_or_null, out, lse, scale, causal, stream)


def fa_fwd_gqa_fp16(q, k, v, mask_or_null, out, lse, scale, causal, stream=None):
    """fp16 grouped-query forward."""
    _fwd_gqa("fa_fwd_gqa_fp16", torch.float16, q, k, v, mask_or_null, out, lse, scale, causal, stream)


# ---------------------------------------------------------------- per-head additive bias
def _fwd_bias(fn_name, dtype, q, k, v, bias, out, lse, scale, causal, stream):
    B, H, N, d = _check(q, k, v, None, out, lse, dtype)
    if (bias is None or bias.dtype != torch.float32 or bias.shape != (B, H, N, N) or not bias.is_contiguous()
            or not bias.is_cuda):
        raise ValueError("bias must be a contiguous CUDA float32 [B, H, N, N] tensor")
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(bias), _ptr(out), _ptr(lse), B, H, N, d, float(scale),
                               int(bool(causal)), ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_fwd_bias(q, k, v, bias, out, lse, scale, causal, stream=None):
    """bf16 forward with a per-head additive bias [B, H, N, N] (fp32)."""
    _fwd_bias("fa_fwd_bias", torch.bfloat16, q, k, v, bias, out, lse, scale, causal, stream)


def fa_fwd_bias_fp16(q, k, v, bias, out, lse, scale, causal, stream=None):
    """fp16 forward with a per-head additive bias [B, H, N, N] (fp32)."""
    _fwd_bias("fa_fwd_bias_fp16", torch.float16, q, k, v, bias, out, lse, scale, causal, stream)


def attention_bias(q, k, v, bias, scale=None, causal=False, stream=None):
    """Forward with a per-head additive bias; allocates O and lse."""
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fn = {torch.bfloat16: fa_fwd_bias, torch.float16: fa_fwd_bias_fp16}[q.dtype]
    fn(q, k, v, bias, out, lse, scale, causal, stream)
    return out, lse


# ---------------------------------------------------------------- split-KV decoding
def fa_splitkv_num_splits(B, H, Nq, Nk, d) -> int:
    n = int(lib.fa_splitkv_num_splits(int(B), int(H), int(Nq), int(Nk), int(d)))
    if n < 0:
        raise FAError(n, "fa_splitkv_num_splits")
    return n


def fa_splitkv_workspace_bytes(B, H, Nq, d, n_splits) -> int:
    n = int(lib.fa_splitkv_workspace_bytes(int(B), int(H), int(Nq), int(d), int(n_splits)))
    if n < 0:
        raise FAError(n, "fa_splitkv_workspace_bytes")
    return n


def _check_splitkv(q, k, v, out, lse, dtype):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape or out.shape != q.shape:
        raise ValueError("q, out must be [B, H, Nq, d] and k, v [B, H, Nk, d]")
    B, H, Nq, d = q.shape
    if k.shape[0] != B or k.shape[1] != H or k.shape[3] != d:
        raise ValueError("k, v must be [B, H, Nk, d] with q's B, H, d")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, Nq):
        raise ValueError("lse must be a contiguous CUDA float32 [B, H, Nq] tensor")
    return B, H, Nq, k.shape[2], d


def _raw_splitkv(fn_name, q, k, v, out, lse, scale, causal, n_splits, workspace, stream, dtype):
    B, H, Nq, Nk, d = _check_splitkv(q, k, v, out, lse, dtype)
    if workspace is None or not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nq, Nk, d, float(scale),
                               int(bool(causal)), int(n_splits), _ptr(workspace), nbytes,
                               ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_fwd_splitkv(q, k, v, out, lse, scale, causal, n_splits, workspace, stream=None):
    """bf16 split-KV forward (Nq <= 16 query rows, Nk keys) into ``out`` and ``lse``."""
    _raw_splitkv("fa_fwd_splitkv", q, k, v, out, lse, scale, causal, n_splits, workspace, stream, torch.bfloat16)


def fa_fwd_splitkv_fp16(q, k, v, out, lse, scale, causal, n_splits, workspace, stream=None):
    """fp16 split-KV forward into ``out`` and ``lse``."""
    _raw_splitkv("fa_fwd_splitkv_fp16", q, k, v, out, lse, scale, causal, n_splits, workspace, stream,
                 torch.float16)


def fa_fwd_splitkv_noalloc(q, k, v, out, lse, scale, causal, n_splits, stream=None):
    """bf16 split-KV forward with no workspace: for callers that cannot allocate
    device memory at the call site (a framework owning all device memory, a
    serving loop that must not pay cudaMalloc's device-wide synchronisation, a
    fixed-budget embedded host). The library's fixed 16 MiB scratch array is
    used instead; calls that overlap on the GPU race on it."""
    B, H, Nq, Nk, d = _check_splitkv(q, k, v, out, lse, torch.bfloat16)
    rc = lib.fa_fwd_splitkv_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Nq, Nk, d, float(scale),
                                    int(bool(causal)), int(n_splits), ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_splitkv_noalloc")


def attention_decode(q, k, v, scale=None, causal=False, n_splits=None, stream=None):
    """Split-KV forward for few query rows; the workspace is a torch allocation."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    n_splits = fa_splitkv_num_splits(B, H, Nq, Nk, d) if n_splits is None else n_splits
    ws = torch.empty(fa_splitkv_workspace_bytes(B, H, Nq, d, n_splits), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    fn = {torch.bfloat16: fa_fwd_splitkv, torch.float16: fa_fwd_splitkv_fp16}[q.dtype]
    fn(q, k, v, out, lse, scale, causal, n_splits, ws, stream)
    return out, lse


# ---------------------------------------------------------------- 8-bit key/value cache
class KVCacheQ8(NamedTuple):
    """A paged cache of K and V in 8 bits: codes [n_pages, Hkv, page, d] (torch.int8 or torch.float8_e4m3fn) and
    scales [n_pages, Hkv] (float32); a value is code * scale. Which pages a sequence owns is the caller's page table."""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


_KVQ8_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}
_FP16_SUFFIX = {torch.bfloat16: "", torch.float16: "_fp16"}


def kv_cache_q8(n_pages, Hkv, page, d, dtype=torch.int8, device="cuda") -> KVCacheQ8:
    """An empty cache of ``n_pages`` pages of ``page`` tokens (16, 32, 64 or 128), codes in ``dtype``."""
    if dtype not in _KVQ8_FORMATS:
        raise ValueError("codes are torch.int8 or torch.float8_e4m3fn")
    codes = [torch.zeros((n_pages, Hkv, page, d), dtype=torch.uint8, device=device).view(dtype) for _ in range(2)]
    scales = [torch.zeros((n_pages, Hkv), dtype=torch.float32, device=device) for _ in range(2)]
    return KVCacheQ8(*codes, *scales)


# The checks below run on every call, in a decoding loop beside kernels of a few microseconds: they ask each tensor as
# little as possible (get_device() is the index, -1 off the GPU).
def _on(index, stream):
    """Context in which device ``index`` is current and torch allocates for ``stream`` (None: the device's current one)."""
    if stream is None:
        current = _get_device() if _get_device is not None else torch.cuda.current_device()
        return _NOTHING if index == current else torch.cuda.device(index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", index))
    if stream.device.index != index:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors are on cuda:{index}")
    return torch.cuda.stream(stream)


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NOTHING = _Nothing()


def _raw_stream(index, stream):
    if stream is None:
        return _get_raw_stream(index) if _get_raw_stream is not None else torch.cuda.current_stream(index).cuda_stream
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


# Contiguous tensors on the current device, past torch's dispatcher where that is possible: 2 us beside a launch where
# torch.empty takes 4 and Tensor.new_empty 6. Dispatch modes do not see them. Under deterministic algorithms torch fills
# what it hands out with NaN; its public function does so here too.
def _empty(shape, strides, dtype):
    if _empty_strided_cuda is None or torch.are_deterministic_algorithms_enabled():
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    return _empty_strided_cuda(shape, strides, dtype)


def _empty4(a, b, c, d, dtype):
    return _empty((a, b, c, d), (b * c * d, c * d, d, 1), dtype)


def _empty3(a, b, c, dtype):
    return _empty((a, b, c), (b * c, c, 1), dtype)


def _empty_bytes(n):
    return _empty((n,), (1,), torch.uint8)


def _check_tensor(name, t, dtype, shape, index):
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")


def _nbytes(workspace, index):
    if workspace is None:
        return 0
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
    return workspace.numel() * workspace.element_size()


_F32, _I32 = torch.float32, torch.int32


def _check_kvq8(cache, page_table):
    """(device index, codes' shape, arguments of the cache for the C call) after checking its tensors against each
    other, and the page table's form."""
    kc, vc, ks, vs = cache
    fmt = _KVQ8_FORMATS.get(kc.dtype)
    shape = kc.shape
    if fmt is None or len(shape) != 4:
        raise ValueError("cache codes must be int8 or float8_e4m3fn tensors [n_pages, Hkv, page, d]")
    index = kc.get_device()
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    table, scales = page_table.shape, shape[:2]
    if not (vc.dtype is kc.dtype and vc.shape == shape and ks.dtype is _F32 and vs.dtype is _F32 and ks.shape == scales
            and vs.shape == scales and page_table.dtype is _I32 and len(table) == 2 and vc.get_device() == index
            and ks.get_device() == index and vs.get_device() == index and page_table.get_device() == index
            and kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and page_table.is_contiguous()):
        if len(table) != 2:
            raise ValueError("page_table must be int32 [nseq, max_pages]")
        for name, t, dtype, want in (("k_codes", kc, kc.dtype, shape), ("v_codes", vc, kc.dtype, shape),
                                     ("k_scale", ks, _F32, scales), ("v_scale", vs, _F32, scales),
                                     ("page_table", page_table, _I32, table)):
            _check_tensor(name, t, dtype, want, index)
    ptrs = (kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), page_table.data_ptr())
    return index, fmt, shape, table, ptrs


def kvq8_append(cache, k, v, page_table, cu_seqlens, cache_lens, max_new, stream=None):
    """Quantise new tokens' ``k``, ``v`` [total, Hkv, d] (bf16 or fp16; any strides of tokens and heads that are
    multiples of 8, rows contiguous) into ``cache``: tokens [cu_seqlens[s], cu_seqlens[s+1]) go to positions
    cache_lens[s], ... of sequence s, at most ``max_new`` per sequence. ``cache_lens`` is left as it is."""
    index, fmt, (n_pages, Hkv, page, d), (nseq, max_pages), cache_ptrs = _check_kvq8(cache, page_table)
    dtype, shape = k.dtype, k.shape
    suffix = _FP16_SUFFIX.get(dtype)
    if suffix is None or len(shape) != 3 or shape[1] != Hkv or shape[2] != d:
        raise ValueError(f"k, v must be bf16 or fp16 tensors [total, {Hkv}, {d}]")
    total = shape[0]
    strides = []
    for name, t in (("k", k), ("v", v)):
        if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
            raise ValueError(f"{name} must be a {dtype} tensor [total, {Hkv}, {d}] on cuda:{index}, k and v alike")
        s0, s1, s2 = t.stride()
        if s2 != 1:
            raise ValueError(f"{name}: the head dimension must be contiguous")
        strides += (s0 if total > 1 else 0, s1 if Hkv > 1 else 0)
    _check_tensor("cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,), index)
    _check_tensor("cache_lens", cache_lens, torch.int32, (nseq,), index)
    name = "fa_kvq8_append" + suffix
    with _on(index, stream):
        rc = getattr(lib, name)(k.data_ptr(), v.data_ptr(), *strides, cu_seqlens.data_ptr(), cache_lens.data_ptr(),
                                nseq, total, int(max_new), *cache_ptrs, n_pages, max_pages, page, Hkv, d, fmt,
                                _raw_stream(index, stream))
    if rc != FA_OK:
        raise FAError(rc, name)


def kvq8_read(cache, page_table, cu_seqlens, total, max_len, first=None, dtype=torch.bfloat16, k=None, v=None,
              stream=None):
    """Cached tokens back as packed K, V [total, Hkv, d]: rows [cu_seqlens[s], cu_seqlens[s+1]) (at most ``max_len``)
    are positions first[s], first[s] + 1, ... of sequence s (``first`` None: from 0). Rows that no sequence covers are
    not written; ``k`` and ``v`` are allocated unless given."""
    index, fmt, (n_pages, Hkv, page, d), (nseq, max_pages), cache_ptrs = _check_kvq8(cache, page_table)
    _check_tensor("cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,), index)
    if first is not None:
        _check_tensor("first", first, torch.int32, (nseq,), index)
    suffix = _FP16_SUFFIX.get(dtype)
    if suffix is None:
        raise ValueError(f"unsupported dtype {dtype}")
    name = "fa_kvq8_read" + suffix
    shape = (int(total), Hkv, d)
    with _on(index, stream):
        k = _empty3(*shape, dtype) if k is None else k
        v = _empty3(*shape, dtype) if v is None else v
        _check_tensor("k", k, dtype, shape, index)
        _check_tensor("v", v, dtype, shape, index)
        rc = getattr(lib, name)(*cache_ptrs, n_pages, max_pages, page, cu_seqlens.data_ptr(),
                                None if first is None else first.data_ptr(), nseq, int(total), int(max_len),
                                k.data_ptr(), v.data_ptr(), Hkv, d, fmt, _raw_stream(index, stream))
    if rc != FA_OK:
        raise FAError(rc, name)
    return k, v


def fa_kvq8_num_parts(B, H, Hkv, Nq, max_len, d) -> int:
    n = int(lib.fa_kvq8_num_parts(int(B), int(H), int(Hkv), int(Nq), int(max_len), int(d)))
    if n < 0:
        raise FAError(n, "fa_kvq8_num_parts")
    return n


def fa_kvq8_workspace_bytes(H, Hkv, Nq, d, n_parts) -> int:
    n = int(lib.fa_kvq8_workspace_bytes(int(H), int(Hkv), int(Nq), int(d), int(n_parts)))
    if n < 0:
        raise FAError(n, "fa_kvq8_workspace_bytes")
    return n


def _raw_kvq8(fn_name, dtype, q, cache, page_table, kv_lens, out, lse, scale, causal, max_len, n_parts, workspace,
              stream):
    """``out``, ``lse`` None: allocated; ``max_len``, ``n_parts``, ``workspace`` None: chosen and allocated."""
    index, fmt, (n_pages, Hkv, page, d), (nseq, max_pages), cache_ptrs = _check_kvq8(cache, page_table)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, H, Nq, d]")
    B, H, Nq, dq = shape
    if dq != d or H % Hkv or nseq != B:
        raise ValueError("q: [B, H, Nq, d] with the cache's d, its Hkv dividing H and one page table row per b")
    _check_tensor("q", q, dtype, shape, index)
    _check_tensor("kv_lens", kv_lens, torch.int32, (B,), index)
    max_len = max_pages * page if max_len is None else int(max_len)
    with _on(index, stream):
        if out is None:
            out = _empty4(B, H, Nq, d, dtype)
            lse = _empty3(B, H, Nq, _F32)
        else:
            _check_tensor("out", out, dtype, shape, index)
            _check_tensor("lse", lse, torch.float32, shape[:3], index)
        n_parts = fa_kvq8_num_parts(B, H, Hkv, Nq, max_len, d) if n_parts is None else int(n_parts)
        if workspace is None and n_parts > 0:
            workspace = _empty_bytes(fa_kvq8_workspace_bytes(H, Hkv, Nq, d, n_parts))
        rc = getattr(lib, fn_name)(q.data_ptr(), *cache_ptrs, n_pages, max_pages, page, kv_lens.data_ptr(),
                                   out.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq, max_len, d, fmt, float(scale), bool(causal),
                                   n_parts, None if workspace is None else workspace.data_ptr(),
                                   _nbytes(workspace, index),
                                   _raw_stream(index, stream))
    if rc != FA_OK:
        raise FAError(rc, fn_name)
    return out, lse


def fa_fwd_kvq8(q, cache, page_table, kv_lens, out, lse, scale, causal, max_len, n_parts, workspace, stream=None):
    """bf16 forward of 1 to 16 query rows per sequence over an 8-bit cache, into ``out`` and ``lse``."""
    _raw_kvq8("fa_fwd_kvq8", torch.bfloat16, q, cache, page_table, kv_lens, out, lse, scale, causal, max_len,
              n_parts, workspace, stream)


def fa_fwd_kvq8_fp16(q, cache, page_table, kv_lens, out, lse, scale, causal, max_len, n_parts, workspace,
                     stream=None):
    """fp16 forward over an 8-bit cache (see ``fa_fwd_kvq8``)."""
    _raw_kvq8("fa_fwd_kvq8_fp16", torch.float16, q, cache, page_table, kv_lens, out, lse, scale, causal, max_len,
              n_parts, workspace, stream)


def attention_kvq8(q, cache, page_table, kv_lens, scale=None, causal=False, max_len=None, n_parts=None, stream=None):
    """O [B, H, Nq, d] and lse [B, H, Nq] of 1 to 16 query rows per sequence over its first kv_lens[b] cached tokens.
    ``max_len`` bounds every length (the page table's reach unless given); the workspace is a torch allocation."""
    suffix = _FP16_SUFFIX.get(q.dtype)
    if suffix is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    return _raw_kvq8("fa_fwd_kvq8" + suffix, q.dtype, q, cache, page_table, kv_lens, None, None, scale, causal, max_len,
                     n_parts, None, stream)


# ---------------------------------------------------------------- packed variable-length batch
def _raw_varlen(fn_name, dtype, q, k, v, out, lse, cu_seqlens, max_seqlen, scale, causal, stream):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor [total, heads, d]")
    total, H, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (total, Hkv, d) or v.shape != k.shape or out.shape != q.shape or H % Hkv:
        raise ValueError("q, out: [total, H, d]; k, v: [total, Hkv, d] with Hkv dividing H")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (H, total):
        raise ValueError("lse must be a contiguous CUDA float32 [H, total] tensor")
    if (cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous()
            or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2):
        raise ValueError("cu_seqlens must be a contiguous CUDA int32 [nseq + 1] tensor")
    nseq = cu_seqlens.numel() - 1
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens), nseq, total,
                               int(max_seqlen), H, Hkv, d, float(scale), int(bool(causal)),
                               ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_fwd_varlen(q, k, v, out, lse, cu_seqlens, max_seqlen, scale, causal, stream=None):
    """bf16 forward over packed sequences: q, out [total, H, d], k, v [total, Hkv, d], lse [H, total]."""
    _raw_varlen("fa_fwd_varlen", torch.bfloat16, q, k, v, out, lse, cu_seqlens, max_seqlen, scale, causal, stream)


def fa_fwd_varlen_fp16(q, k, v, out, lse, cu_seqlens, max_seqlen, scale, causal, stream=None):
    """fp16 forward over packed sequences."""
    _raw_varlen("fa_fwd_varlen_fp16", torch.float16, q, k, v, out, lse, cu_seqlens, max_seqlen, scale, causal,
                stream)


def attention_varlen(q, k, v, cu_seqlens, max_seqlen, scale=None, causal=False, stream=None):
    """O [total, H, d] and lse [H, total] for packed sequences; allocates the outputs with torch."""
    total, H, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q)
    lse = torch.empty((H, total), dtype=torch.float32, device=q.device)
    fn = {torch.bfloat16: fa_fwd_varlen, torch.float16: fa_fwd_varlen_fp16}[q.dtype]
    fn(q, k, v, out, lse, cu_seqlens, max_seqlen, scale, causal, stream)
    return out, lse


# ---------------------------------------------------------------- backward (recomputation)
def fa_bwd_workspace_bytes(B, H, N, d) -> int:
    n = int(lib.fa_bwd_workspace_bytes(int(B), int(H), int(N), int(d)))
    if n < 0:
        raise FAError(n, "fa_bwd_workspace_bytes")
    return n


def _raw_bwd(fn_name, dtype, q, k, v, out, dout, lse, dq, dk, dv, scale, causal, workspace, stream):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout), ("dq", dq), ("dk", dk),
                    ("dv", dv)):
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
        if t.dim() != 4 or t.shape != q.shape:
            raise ValueError(f"{name} must be [B, H, N, d] like q")
    B, H, N, d = q.shape
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, N):
        raise ValueError("lse must be a contiguous CUDA float32 [B, H, N] tensor")
    if workspace is None or not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    rc = getattr(lib, fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, H, N, d, float(scale), int(bool(causal)), _ptr(workspace), nbytes,
                               ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, fn_name)


def fa_bwd(q, k, v, out, dout, lse, dq, dk, dv, scale, causal, workspace, stream=None):
    """bf16 backward into caller-provided ``dq``, ``dk``, ``dv`` [B,H,N,d]."""
    _raw_bwd("fa_bwd", torch.bfloat16, q, k, v, out, dout, lse, dq, dk, dv, scale, causal, workspace, stream)


def fa_bwd_fp16(q, k, v, out, dout, lse, dq, dk, dv, scale, causal, workspace, stream=None):
    """fp16 backward into caller-provided ``dq``, ``dk``, ``dv``."""
    _raw_bwd("fa_bwd_fp16", torch.float16, q, k, v, out, dout, lse, dq, dk, dv, scale, causal, workspace, stream)


def attention_backward(q, k, v, out, dout, lse, scale=None, causal=False, workspace=None, stream=None):
    """(dq, dk, dv) of sum(dout * out) for out, lse from ``attention``; allocates
    the outputs and, unless given, the workspace with torch."""
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if workspace is None:
        workspace = torch.empty(fa_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fn = {torch.bfloat16: fa_bwd, torch.float16: fa_bwd_fp16}[q.dtype]
    fn(q, k, v, out, dout, lse, dq, dk, dv, scale, causal, workspace, stream)
    return dq, dk, dv


# ---------------------------------------------------------------- keys of another sequence
def fa_cross_num_splits(B, H, Nq, Nk) -> int:
    n = int(lib.fa_cross_num_splits(int(B), int(H), int(Nq), int(Nk)))
    if n < 0:
        raise FAError(n, "fa_cross_num_splits")
    return n


def _check_cross(q, k, v, kv_lens, dtype):
    """(device index, B, H, Hkv, Nq, Nk, d) after checking the inputs."""
    sq, sk = q.shape, k.shape
    if len(sq) != 4 or len(sk) != 4:
        raise ValueError("q must be [B, H, Nq, d] and k, v [B, Hkv, Nk, d]")
    B, H, Nq, d = sq
    Hkv, Nk = sk[1], sk[2]
    if sk[0] != B or sk[3] != d or Hkv < 1 or H % Hkv:
        raise ValueError("k, v must be [B, Hkv, Nk, d] with q's B and d, and Hkv dividing H")
    index = q.get_device()
    if index < 0:
        raise ValueError("q must be on a CUDA device")
    _check_tensor("q", q, dtype, sq, index)
    _check_tensor("k", k, dtype, sk, index)
    _check_tensor("v", v, dtype, sk, index)
    if kv_lens is not None:
        _check_tensor("kv_lens", kv_lens, torch.int32, (B,), index)
    return index, B, H, Hkv, Nq, Nk, d


def _raw_cross(fn_name, dtype, q, k, v, kv_lens, out, lse, scale, n_splits, workspace, stream):
    """``out``, ``lse`` None: allocated; ``n_splits`` None: chosen, with a workspace from torch."""
    index, B, H, Hkv, Nq, Nk, d = _check_cross(q, k, v, kv_lens, dtype)
    with _on(index, stream):
        if out is None:
            out = _empty4(B, H, Nq, d, dtype)
            lse = _empty3(B, H, Nq, _F32)
            n_splits = fa_cross_num_splits(B, H, Nq, Nk) if n_splits is None else n_splits
            if n_splits > 1:
                workspace = _empty_bytes(fa_splitkv_workspace_bytes(B, H, Nq, d, n_splits))
        else:
            _check_tensor("out", out, dtype, q.shape, index)
            _check_tensor("lse", lse, torch.float32, (B, H, Nq), index)
        rc = getattr(lib, fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                   None if kv_lens is None else kv_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H,
                                   Hkv, Nq, Nk, d, float(scale), int(n_splits),
                                   None if workspace is None else workspace.data_ptr(), _nbytes(workspace, index),
                                   _raw_stream(index, stream))
    if rc != FA_OK:
        raise FAError(rc, fn_name)
    return out, lse


def fa_fwd_cross(q, k, v, kv_lens, out, lse, scale, n_splits=1, workspace=None, stream=None):
    """bf16 forward of q [B, H, Nq, d] over k, v [B, Hkv, Nk, d]; batch index b uses its first kv_lens[b] keys
    (int32 [B]; None: all), whatever lies behind them. ``workspace`` as for ``fa_fwd_splitkv`` when n_splits > 1."""
    _raw_cross("fa_fwd_cross", torch.bfloat16, q, k, v, kv_lens, out, lse, scale, n_splits, workspace, stream)


def fa_fwd_cross_fp16(q, k, v, kv_lens, out, lse, scale, n_splits=1, workspace=None, stream=None):
    """fp16 forward over keys of another length (see ``fa_fwd_cross``)."""
    _raw_cross("fa_fwd_cross_fp16", torch.float16, q, k, v, kv_lens, out, lse, scale, n_splits, workspace, stream)


def attention_cross(q, k, v, kv_lens=None, scale=None, n_splits=None, stream=None):
    """O [B, H, Nq, d] and lse [B, H, Nq] of queries over the keys of another sequence; allocates the outputs and, when
    the keys are split, the workspace."""
    suffix = _FP16_SUFFIX.get(q.dtype)
    if suffix is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    return _raw_cross("fa_fwd_cross" + suffix, q.dtype, q, k, v, kv_lens, None, None, scale, n_splits, None, stream)


def fa_bwd_cross_workspace_bytes(B, H, Hkv, Nq, Nk, d) -> int:
    n = int(lib.fa_bwd_cross_workspace_bytes(int(B), int(H), int(Hkv), int(Nq), int(Nk), int(d)))
    if n < 0:
        raise FAError(n, "fa_bwd_cross_workspace_bytes")
    return n


def _raw_bwd_cross(fn_name, dtype, q, k, v, kv_lens, out, dout, lse, dq, dk, dv, scale, workspace, stream):
    """``dq``, ``dk``, ``dv`` None: allocated; ``workspace`` None: allocated."""
    index, B, H, Hkv, Nq, Nk, d = _check_cross(q, k, v, kv_lens, dtype)
    _check_tensor("out", out, dtype, q.shape, index)
    _check_tensor("dout", dout, dtype, q.shape, index)
    _check_tensor("lse", lse, torch.float32, (B, H, Nq), index)
    with _on(index, stream):
        if workspace is None:
            workspace = _empty_bytes(fa_bwd_cross_workspace_bytes(B, H, Hkv, Nq, Nk, d))
        if dq is None:
            dq = _empty4(B, H, Nq, d, dtype)
            dk, dv = _empty4(B, Hkv, Nk, d, dtype), _empty4(B, Hkv, Nk, d, dtype)
        else:
            _check_tensor("dq", dq, dtype, q.shape, index)
            _check_tensor("dk", dk, dtype, k.shape, index)
            _check_tensor("dv", dv, dtype, k.shape, index)
        rc = getattr(lib, fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                   None if kv_lens is None else kv_lens.data_ptr(), out.data_ptr(), dout.data_ptr(),
                                   lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Hkv, Nq, Nk, d,
                                   float(scale), workspace.data_ptr(), _nbytes(workspace, index),
                                   _raw_stream(index, stream))
    if rc != FA_OK:
        raise FAError(rc, fn_name)
    return dq, dk, dv


def fa_bwd_cross(q, k, v, kv_lens, out, dout, lse, dq, dk, dv, scale, workspace, stream=None):
    """bf16 gradients of ``fa_fwd_cross`` into ``dq`` (like q) and ``dk``, ``dv`` (like k, summed over the query heads
    that share them; 0 past kv_lens); ``workspace`` of
    ``fa_bwd_cross_workspace_bytes(B, H, Hkv, Nq, Nk, d)`` bytes."""
    _raw_bwd_cross("fa_bwd_cross", torch.bfloat16, q, k, v, kv_lens, out, dout, lse, dq, dk, dv, scale, workspace, stream)


def fa_bwd_cross_fp16(q, k, v, kv_lens, out, dout, lse, dq, dk, dv, scale, workspace, stream=None):
    """fp16 gradients of ``fa_fwd_cross_fp16`` (see ``fa_bwd_cross``)."""
    _raw_bwd_cross("fa_bwd_cross_fp16", torch.float16, q, k, v, kv_lens, out, dout, lse, dq, dk, dv, scale, workspace,
                   stream)


def attention_cross_backward(q, k, v, out, dout, lse, kv_lens=None, scale=None, workspace=None, stream=None):
    """(dq, dk, dv) of sum(dout * out) for out, lse from ``attention_cross``; allocates the outputs and, unless given,
    the workspace with torch."""
    suffix = _FP16_SUFFIX.get(q.dtype)
    if suffix is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    return _raw_bwd_cross("fa_bwd_cross" + suffix, q.dtype, q, k, v, kv_lens, out, dout, lse, None, None, None, scale,
                          workspace, stream)


def fa_get_device_status(stream=None) -> int:
    return int(lib.fa_get_device_status(ctypes.c_void_p(_stream_handle(stream))))


def fa_selftest_wait_timeout(timeout_ns, stream=None):
    """Enqueue the bounded-wait self-test (a wait nothing completes); afterwards
    fa_get_device_status() must report FA_ERR_TIMEOUT."""
    rc = lib.fa_selftest_wait_timeout(int(timeout_ns), ctypes.c_void_p(_stream_handle(stream)))
    if rc != FA_OK:
        raise FAError(rc, "fa_selftest_wait_timeout")


def fa_num_sms() -> int:
    return int(lib.fa_num_sms())
