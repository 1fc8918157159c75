"""Python binding of the low-rank adapters of many requests (include/lora.h) of
libw4a16.so.

Argument marshalling only; there is no fallback, and no gradient: the call is not part of
torch's autograd graph.  base is what w4a16_gemm, fp8.fp8_gemm or another product gave for
the rows x, or for the quantised rows (x, xs) of rowquant.rmsnorm_quantize_rows and
swiglu_quantize_rows with kind "fp8".
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import (_bad, _check, _empty_on, _keep_bytes, _launch_stream, _require,
               _require_workspace, _scratch, _used_on, load_library)

C_FUNCTIONS_LORA = ("lora_workspace_bytes", "lora_add")
_FLAGS = {torch.float16: 0x0, torch.bfloat16: 0x1}
_X_FP8 = 0x10
_CODES = (torch.float8_e4m3fn, torch.uint8)

_declared = None
_ws_bytes = {}


def _lib():
    global _declared
    if _declared is None:
        lib = load_library()
        p, i64, u32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
        lib.lora_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, u32]
        lib.lora_workspace_bytes.restype = sz
        lib.lora_add.argtypes = [p, i64, p, i64, p, p, p, p, p, p, i64, i64, i64, i64, i64, i64, u32,
                                 p, sz, p]
        lib.lora_add.restype = ctypes.c_int
        _declared = lib
    return _declared


def lora_workspace_bytes(M: int, N: int, K: int, R: int, L: int, flags: int) -> int:
    return int(_lib().lora_workspace_bytes(M, N, K, R, L, flags))


def _rows(t: torch.Tensor, where: str, name: str, dtypes) -> int:
    """Checks a [M][W] tensor of rows; returns their distance in elements."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        _bad(f"{where}: {name}: need a [rows][columns] device tensor of {dtypes}, got {t.dtype} "
             f"{tuple(t.shape)} on {t.device}")
    M, W = t.shape
    ld = t.stride(0) if M > 1 else W   # the stride of a single row is never used
    if (t.stride(1) != 1 and W > 1) or ld < W:
        _bad(f"{where}: {name}: rows must be contiguous and not overlap")
    return ld


def lora_add(base: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
             ids: torch.Tensor, scale: Optional[torch.Tensor] = None,
             xs: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [M][N] = base + scale[ids] * (x a[ids]^T) b[ids]^T, row by row.
    base fp16/bf16 [M][N]; x [M][K] in base's dtype, or E4M3 with xs float32 [M][ceil(K/128)];
    a [L][R][K] and b [L][N][R] in base's dtype; ids int32 [M], a row whose id is outside
    [0, L) has no adapter (out = base); scale float32 [L].  Rows of base, x and out may be
    strided.  out, if given, is the tensor to write: base itself, or one that overlaps no
    input."""
    where = "lora_add"
    dt = base.dtype
    if dt not in _FLAGS:
        _bad(f"{where}: base must be fp16 or bf16")
    ldb = _rows(base, where, "base", (dt,))
    M, N = base.shape
    flags = _FLAGS[dt]
    if xs is None:
        ldx = _rows(x, where, "x", (dt,))
    else:
        flags |= _X_FP8
        ldx = _rows(x, where, "x", _CODES)
    K, dev = x.shape[1], base.get_device()
    if x.shape[0] != M or x.get_device() != dev:
        _bad(f"{where}: x is {tuple(x.shape)} on {x.device}, base {tuple(base.shape)} on "
             f"{base.device}")
    if a.dim() != 3 or b.dim() != 3:
        _bad(f"{where}: a and b must be [L][R][K] and [L][N][R]")
    L, R = a.shape[:2]
    if a.shape[2] != K or tuple(b.shape) != (L, N, R):
        _bad(f"{where}: a is {tuple(a.shape)}, b {tuple(b.shape)}, base {tuple(base.shape)}, "
             f"x {tuple(x.shape)}")
    if not (a.dtype == b.dtype == dt and ids.dtype == torch.int32 and ids.numel() == M
            and a.is_contiguous() and b.is_contiguous() and ids.is_contiguous()
            and a.get_device() == b.get_device() == ids.get_device() == dev):
        _require(a, f"{where}: a", dt, L * R * K, base.device)       # one of them raises with the
        _require(b, f"{where}: b", dt, L * N * R, base.device)       # details
        _require(ids, f"{where}: ids", torch.int32, M, base.device)
    if scale is not None:
        _require(scale, f"{where}: scale", torch.float32, L, base.device)
    if xs is not None:
        kb = -(-K // 128)
        _require(xs, f"{where}: xs", torch.float32, M * kb, base.device)
        if xs.dim() > 1 and xs.size(-1) != kb:
            _bad(f"{where}: xs is {tuple(xs.shape)}, its rows must hold {kb} scales")
    if out is None:
        # empty_like: 1.2 us where empty with a shape and a device takes 1.7
        out = (torch.empty_like(base) if stream is None and base.is_contiguous()
               else _empty_on(stream, (M, N), dt, base.device))
        ldo = N
    else:
        ldo = _rows(out, where, "out", (dt,))
        if tuple(out.shape) != (M, N) or out.get_device() != dev:
            _bad(f"{where}: out is {tuple(out.shape)} on {out.device}")
    handle = _launch_stream(where, stream, dev)
    if workspace is None:
        key = (M, N, K, R, L, flags)
        need = _ws_bytes.get(key)
        if need is None:
            need = _keep_bytes(_ws_bytes, key, lora_workspace_bytes(M, N, K, R, L, flags))
        if need:
            workspace = _scratch(need, base.device, stream, handle)
    else:
        _require_workspace(workspace, where, dev)
    _check(_lib().lora_add(base.data_ptr(), ldb, x.data_ptr(), ldx,
                           None if xs is None else xs.data_ptr(), a.data_ptr(), b.data_ptr(),
                           None if scale is None else scale.data_ptr(), ids.data_ptr(),
                           out.data_ptr(), ldo, M, N, K, R, L, flags,
                           None if workspace is None else workspace.data_ptr(),
                           0 if workspace is None else workspace.numel() * workspace.element_size(),
                           handle), where)
    if stream is not None:
        _used_on(stream, base, x, xs, a, b, scale, ids, out, workspace)
    return out
