"""Python binding of the fused producers of quantised rows (include/rowquant.h) of
libw4a16.so: the RMS norm and the gated activation, ending in the rows that the
library's products read.

    kind     rows q                     scales s                     product
    "fp8"    float8_e4m3fn [T][W]       float32 [T][ceil(W/128)]     fp8.fp8_gemm
    "int8"   int8 [T][W]                float32 [T]                  w4a8.w4a8_gemm
    "mx"     uint8 [T][W] (E4M3)        uint8 [T][W/32] (E8M0)       mxfp4.mxfp4_gemm
    "x16"    the inputs' dtype [T][W]   None                         w4a16_gemm

Argument marshalling only; there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import (W4A16Error, W4A16_ERR_UNSUPPORTED, _bad, _check, _empty_on, _require,
               _stream_handle, _used_on, load_library)

C_FUNCTIONS_ROWQUANT = ("rowquant_rmsnorm", "rowquant_swiglu")

_F16, _BF16 = torch.float16, torch.bfloat16
# kind -> flag, dtype of q (None: the inputs'), dtype of s, the widths W must divide by
_KINDS = {"fp8": (0x00, torch.float8_e4m3fn, torch.float32, 16),
          "int8": (0x10, torch.int8, torch.float32, 16),
          "mx": (0x20, torch.uint8, torch.uint8, 32),
          "x16": (0x30, None, None, 16)}

_declared = None


def _lib():
    global _declared
    if _declared is None:
        lib = load_library()
        p, i64, u32, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
        lib.rowquant_rmsnorm.argtypes = [p, i64, p, i64, p, f, p, p, p, i64, i64, u32, p]
        lib.rowquant_rmsnorm.restype = ctypes.c_int
        lib.rowquant_swiglu.argtypes = [p, i64, p, i64, p, p, i64, i64, u32, p]
        lib.rowquant_swiglu.restype = ctypes.c_int
        _declared = lib
    return _declared


def _input(t: torch.Tensor, where: str, name: str):
    """Checks an input of rows; returns (T, W, row stride in elements)."""
    if t.dim() != 2 or (t.dtype != _BF16 and t.dtype != _F16) or not t.is_cuda:
        _bad(f"{where}: {name}: need an fp16/bf16 [T][W] device tensor")
    T, W = t.shape
    ld = t.stride(0) if T > 1 else W   # the stride of a single row is never used
    if (t.stride(1) != 1 and W > 1) or ld < W or ld % 8 or t.data_ptr() % 16:
        _bad(f"{where}: {name}: rows must be contiguous, 16-byte aligned and a multiple of 8 "
             "elements apart")
    return T, W, ld


def _same(t: torch.Tensor, like: torch.Tensor, where: str, name: str) -> int:
    """Checks an input that goes with `like`; returns its row stride."""
    if t.shape != like.shape or t.dtype != like.dtype or t.get_device() != like.get_device():
        _bad(f"{where}: {name}: {t.dtype} {tuple(t.shape)} on {t.device} does not go with "
             f"{like.dtype} {tuple(like.shape)} on {like.device}")
    return _input(t, where, name)[2]


def _outputs(where: str, like: torch.Tensor, T: int, W: int, kind: str, q, s, stream):
    """The output tensors (made if not given) and the call's flags."""
    spec = _KINDS.get(kind)
    if spec is None:
        raise ValueError(f"bad kind {kind!r}")
    flag, q_dtype, s_dtype, step = spec
    if W < 1 or W % step:
        raise W4A16Error(W4A16_ERR_UNSUPPORTED, f"{where}: row of {W} elements")
    if q_dtype is None:
        q_dtype = like.dtype
    if q is None:
        # empty_like: 1.2 us where empty with a shape and a device takes 1.7
        q = (torch.empty_like(like, dtype=q_dtype) if stream is None and like.is_contiguous()
             else _empty_on(stream, (T, W), q_dtype, like.device))
    else:
        _require(q, f"{where}: q", q_dtype, T * W, like.device)
    if s_dtype is None:
        if s is not None:
            _bad(f"{where}: kind {kind} has no scales")
    else:
        shape = (T, -(-W // 128)) if kind == "fp8" else (T, W // 32) if kind == "mx" else (T,)
        if s is None:
            s = _empty_on(stream, shape, s_dtype, like.device)
        else:
            _require(s, f"{where}: s", s_dtype, T * (shape[1] if len(shape) == 2 else 1),
                     like.device)
            if len(shape) == 2 and s.dim() > 1 and s.size(-1) != shape[1]:
                _bad(f"{where}: s is {tuple(s.shape)}, its rows must hold {shape[1]} scales")
    return q, s, flag | (0x1 if like.dtype == _BF16 else 0x0)


def rmsnorm_quantize_rows(x: torch.Tensor, weight: torch.Tensor,
                          residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          kind: str = "fp8", q: Optional[torch.Tensor] = None,
                          s: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                          stream=None):
    """(q, s, h): the rows of rms_norm(x + residual) * weight quantised per `kind`, and
    h = x + residual in x's dtype (None without a residual).  x and residual fp16/bf16
    [T][W] (rows may be strided), weight [W].  The norm is taken of the unrounded sum.
    q, s and h, if given, are the contiguous tensors to write."""
    where = "rmsnorm_quantize_rows"
    T, W, ldx = _input(x, where, "x")
    ldr = W if residual is None else _same(residual, x, where, "residual")
    if (weight.dtype != x.dtype or weight.numel() != W or not weight.is_contiguous()
            or weight.get_device() != x.get_device()):
        _require(weight, f"{where}: weight", x.dtype, W, x.device)   # raises with the details
    q, s, flags = _outputs(where, x, T, W, kind, q, s, stream)
    if h is not None:
        _require(h, f"{where}: h", x.dtype, T * W, x.device)
    elif residual is not None:
        h = (torch.empty_like(x) if stream is None and x.is_contiguous()
             else _empty_on(stream, (T, W), x.dtype, x.device))
    _check(_lib().rowquant_rmsnorm(x.data_ptr(), ldx,
                                   None if residual is None else residual.data_ptr(), ldr,
                                   weight.data_ptr(), eps, None if h is None else h.data_ptr(),
                                   q.data_ptr(), None if s is None else s.data_ptr(), T, W, flags,
                                   _stream_handle(stream)), where)
    if stream is not None:
        _used_on(stream, x, residual, weight, q, s, h)
    return q, s, h


def swiglu_quantize_rows(gate: torch.Tensor, up: torch.Tensor, kind: str = "fp8",
                         q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                         stream=None):
    """(q, s): the rows of silu(gate) * up quantised per `kind`.  gate and up fp16/bf16
    [T][W]; rows may be strided, so the halves of one [T][2W] product serve as they are."""
    where = "swiglu_quantize_rows"
    T, W, ldg = _input(gate, where, "gate")
    ldu = _same(up, gate, where, "up")
    q, s, flags = _outputs(where, gate, T, W, kind, q, s, stream)
    _check(_lib().rowquant_swiglu(gate.data_ptr(), ldg, up.data_ptr(), ldu, q.data_ptr(),
                                  None if s is None else s.data_ptr(), T, W, flags,
                                  _stream_handle(stream)), where)
    if stream is not None:
        _used_on(stream, gate, up, q, s)
    return q, s
