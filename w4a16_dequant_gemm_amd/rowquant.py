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

from . import (W4A16Error, W4A16_ERR_UNSUPPORTED, _bad, _check, _ptr, _require, _stream,
               load_library)

ROWQUANT_KIND = {"fp8": 0x00, "int8": 0x10, "mx": 0x20, "x16": 0x30}
ROWQUANT_MAX_ROW = 131072
C_FUNCTIONS_ROWQUANT = ("rowquant_rmsnorm", "rowquant_swiglu")

_declared = False


def _lib():
    global _declared
    lib = load_library()
    if not _declared:
        p, i64, u32, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
        lib.rowquant_rmsnorm.argtypes = [p, i64, p, i64, p, f, p, p, p, i64, i64, u32, p]
        lib.rowquant_rmsnorm.restype = ctypes.c_int
        lib.rowquant_swiglu.argtypes = [p, i64, p, i64, p, p, i64, i64, u32, p]
        lib.rowquant_swiglu.restype = ctypes.c_int
        _declared = True
    return lib


def _input(t: torch.Tensor, where: str, like: Optional[torch.Tensor] = None) -> int:
    """Checks an input of rows; returns its row stride in elements."""
    if t.dim() != 2 or t.dtype not in (torch.float16, torch.bfloat16) or not t.is_cuda:
        _bad(f"{where}: need an fp16/bf16 [T][W] device tensor")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype
                             or t.device != like.device):
        _bad(f"{where}: {t.dtype} {tuple(t.shape)} on {t.device} does not go with {like.dtype} "
             f"{tuple(like.shape)} on {like.device}")
    T, W = t.shape
    if T <= 1:
        ld = W   # one row: its stride is never used
    else:
        ld = t.stride(0)
    if (W > 1 and t.stride(1) != 1) or ld < W or ld % 8 or t.data_ptr() % 16:
        _bad(f"{where}: rows must be contiguous, 16-byte aligned and a multiple of 8 elements "
             "apart")
    return ld


def _outputs(where: str, like: torch.Tensor, kind: str, q, s):
    """The output tensors (made if not given) and the call's flags."""
    if kind not in ROWQUANT_KIND:
        raise ValueError(f"bad kind {kind!r}")
    T, W = like.shape
    if W < 1 or W % (32 if kind == "mx" else 16):
        raise W4A16Error(W4A16_ERR_UNSUPPORTED, f"{where}: row of {W} elements")
    q_dtype, s_dtype, s_shape = {
        "fp8": (torch.float8_e4m3fn, torch.float32, (T, -(-W // 128))),
        "int8": (torch.int8, torch.float32, (T,)),
        "mx": (torch.uint8, torch.uint8, (T, W // 32)),
        "x16": (like.dtype, None, None)}[kind]
    if q is None:
        q = torch.empty((T, W), dtype=q_dtype, device=like.device)
    _require(q, f"{where}: q", q_dtype, T * W, like.device)
    if s_dtype is None:
        if s is not None:
            _bad(f"{where}: kind {kind} has no scales")
    else:
        if s is None:
            s = torch.empty(s_shape, dtype=s_dtype, device=like.device)
        n = 1
        for d in s_shape:
            n *= d
        _require(s, f"{where}: s", s_dtype, n, like.device)
    return q, s, ROWQUANT_KIND[kind] | (0x1 if like.dtype == torch.bfloat16 else 0x0)


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
    ldx = _input(x, f"{where}: x")
    T, W = x.shape
    ldr = W if residual is None else _input(residual, f"{where}: residual", x)
    _require(weight, f"{where}: weight", x.dtype, W, x.device)
    q, s, flags = _outputs(where, x, kind, q, s)
    if residual is not None and h is None:
        h = torch.empty((T, W), dtype=x.dtype, device=x.device)
    if h is not None:
        _require(h, f"{where}: h", x.dtype, T * W, x.device)
    _check(_lib().rowquant_rmsnorm(_ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), eps, _ptr(h),
                                   _ptr(q), _ptr(s), T, W, flags, _stream(stream)), where)
    return q, s, h


def swiglu_quantize_rows(gate: torch.Tensor, up: torch.Tensor, kind: str = "fp8",
                         q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                         stream=None):
    """(q, s): the rows of silu(gate) * up quantised per `kind`.  gate and up fp16/bf16
    [T][W]; rows may be strided, so the halves of one [T][2W] product serve as they are."""
    where = "swiglu_quantize_rows"
    ldg = _input(gate, f"{where}: gate")
    ldu = _input(up, f"{where}: up", gate)
    T, W = gate.shape
    q, s, flags = _outputs(where, gate, kind, q, s)
    _check(_lib().rowquant_swiglu(_ptr(gate), ldg, _ptr(up), ldu, _ptr(q), _ptr(s), T, W, flags,
                                  _stream(stream)), where)
    return q, s
