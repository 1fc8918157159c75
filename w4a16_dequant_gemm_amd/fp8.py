"""Python binding of the block-scaled fp8 entry points (include/fp8.h) of libw4a16.so.

Argument marshalling only: the repack and the products run in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  There is no
fallback.

The rows that fp8_gemm and fp8_grouped_gemm multiply are those of
rowquant.rmsnorm_quantize_rows and rowquant.swiglu_quantize_rows with kind "fp8".
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import (W4A16Error, W4A16_ERR_INVALID_ARG, W4A16_ERR_UNSUPPORTED, W4A16_PLAN_PARAM_SHIFT,
               _bad, _check, _empty_on, _keep_bytes, _ptr, _require, _require_workspace, _stream,
               _stream_handle, _used_on, _workspace_at, load_library)

FP8_LAYOUT_VERSION = 1   # of include/fp8.h
FP8_BLOCK = 128
FP8_PLAN = {"stream": 0x10, "tiled": 0x20}
C_FUNCTIONS_FP8 = ("fp8_packed_bytes", "fp8_repack", "fp8_workspace_bytes", "fp8_gemm",
                   "fp8_grouped_gemm")
_DT = {"fp16": (0x0, torch.float16), "bf16": (0x1, torch.bfloat16)}
_CODES = (torch.float8_e4m3fn, torch.uint8)

_declared = None
_ws_bytes = {}


def _lib():
    global _declared
    if _declared is None:
        lib = load_library()
        p, i64, ci, u32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32,
                               ctypes.c_size_t)
        lib.fp8_packed_bytes.argtypes = [i64, i64, i64]
        lib.fp8_packed_bytes.restype = sz
        lib.fp8_repack.argtypes = [p, p, i64, i64, i64, p, sz, p]
        lib.fp8_repack.restype = ci
        lib.fp8_workspace_bytes.argtypes = [i64, i64, i64, u32]
        lib.fp8_workspace_bytes.restype = sz
        lib.fp8_gemm.argtypes = [p, p, p, sz, p, i64, i64, i64, u32, p, sz, p]
        lib.fp8_gemm.restype = ci
        lib.fp8_grouped_gemm.argtypes = [p, p, p, sz, p, p, p, i64, i64, i64, i64, i64, u32, p]
        lib.fp8_grouped_gemm.restype = ci
        _declared = lib
    return _declared


def plan_flags_fp8(plan) -> int:
    """None, "stream", "tiled", or (name, parameter)."""
    if plan is None:
        return 0
    name, param = (plan, 0) if isinstance(plan, str) else plan
    if name not in FP8_PLAN or not 0 <= int(param) <= 255:
        raise ValueError(f"bad plan hint {plan!r}")
    return FP8_PLAN[name] | (int(param) << W4A16_PLAN_PARAM_SHIFT)


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


@dataclass
class PackedFP8:
    """A repacked fp8 blob and the shape it was made for."""
    data: torch.Tensor   # uint8 device tensor
    E: int               # experts
    K: int
    N: int
    grouped: bool        # made from [E][N][K] (a stack of experts) or [N][K]
    layout_version: int = FP8_LAYOUT_VERSION   # of the library that made it


def fp8_packed_bytes(E: int, K: int, N: int) -> int:
    return int(_lib().fp8_packed_bytes(E, K, N))


def fp8_workspace_bytes(M: int, N: int, K: int, flags: int = 0) -> int:
    return int(_lib().fp8_workspace_bytes(M, N, K, flags))


def fp8_repack(w: torch.Tensor, ws: torch.Tensor, stream=None) -> PackedFP8:
    """w E4M3 [N][K] with ws float32 [ceil(N/128)][ceil(K/128)], or the same with a
    leading dimension of experts -> PackedFP8."""
    if w.dim() not in (2, 3) or w.dtype not in _CODES or not w.is_contiguous() or not w.is_cuda:
        _bad("fp8_repack: w must be a contiguous E4M3 device tensor [N][K] or [E][N][K]")
    E = w.shape[0] if w.dim() == 3 else 1
    N, K = w.shape[-2:]
    if ws.shape != (*w.shape[:-2], _blocks(N), _blocks(K)):
        _bad(f"fp8_repack: ws is {tuple(ws.shape)}, w {tuple(w.shape)}")
    nbytes = fp8_packed_bytes(E, K, N)
    if nbytes == 0:
        raise W4A16Error(W4A16_ERR_UNSUPPORTED if K % 16 else W4A16_ERR_INVALID_ARG,
                         "fp8_packed_bytes")
    _require(ws, "fp8_repack: ws", torch.float32, E * _blocks(N) * _blocks(K), w.device)
    packed = _empty_on(stream, nbytes, torch.uint8, w.device)
    _check(_lib().fp8_repack(_ptr(w), _ptr(ws), E, K, N, _ptr(packed), nbytes, _stream(stream)),
           "fp8_repack")
    if stream is not None:
        _used_on(stream, w, ws)
    return PackedFP8(packed, E, K, N, w.dim() == 3)


def _rows(where: str, xq: torch.Tensor, xs: torch.Tensor, packed: PackedFP8, out: str):
    if xq.dim() != 2 or xq.dtype not in _CODES or not xq.is_cuda or not xq.is_contiguous():
        _bad(f"{where}: xq must be a contiguous E4M3 [rows][K] device tensor")
    if packed.layout_version != FP8_LAYOUT_VERSION:
        _bad(f"{where}: blob layout version {packed.layout_version}, library {FP8_LAYOUT_VERSION}")
    rows, K = xq.shape
    if K != packed.K:
        _bad(f"{where}: xq has K = {K}, the blob {packed.K}")
    if out not in _DT:
        raise ValueError(f"bad output dtype {out!r}")
    dev = xq.get_device()
    kb = _blocks(K)
    if (xs.dtype != torch.float32 or xs.numel() != rows * kb or not xs.is_contiguous()
            or xs.get_device() != dev):
        _require(xs, f"{where}: xs", torch.float32, rows * kb, xq.device)   # raises
    # the same numbers the other way round, a row of scales per block, give another product
    if xs.dim() > 1 and xs.size(-1) != kb:
        _bad(f"{where}: xs is {tuple(xs.shape)}, its rows must hold {kb} scales")
    if packed.data.get_device() != dev:
        _bad(f"{where}: the blob is on another device")
    return rows, K, *_DT[out]


def _workspace_need(device_index: int, M: int, N: int, K: int, flags: int) -> int:
    key = (device_index, M, N, K, flags)
    need = _ws_bytes.get(key)
    if need is None:
        need = _keep_bytes(_ws_bytes, key, fp8_workspace_bytes(M, N, K, flags))
    return need


def fp8_gemm(xq: torch.Tensor, xs: torch.Tensor, packed: PackedFP8, out: str = "bf16",
             Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             plan=None, stream=None) -> torch.Tensor:
    """Y [M][N] (fp16 or bf16 per `out`) = rows xq [M][K] with scales xs [M][ceil(K/128)]
    times the blob's weights."""
    M, K, flag, tdt = _rows("fp8_gemm", xq, xs, packed, out)
    if packed.grouped:
        _bad("fp8_gemm: the blob holds experts")
    N = packed.N
    if Y is None:
        Y = (torch.empty((M, N), dtype=tdt, device=xq.device) if stream is None
             else _empty_on(stream, (M, N), tdt, xq.device))
    else:
        _require(Y, "fp8_gemm: Y", tdt, M * N, xq.device)
    flags = flag if plan is None else flag | plan_flags_fp8(plan)
    dev, handle = xq.get_device(), _stream_handle(stream)
    if workspace is None:
        need = _workspace_need(dev, M, N, K, flags)
        if need:
            workspace = _workspace_at(need, dev, handle)
    else:
        _require_workspace(workspace, "fp8_gemm", dev)
    _check(_lib().fp8_gemm(xq.data_ptr(), xs.data_ptr(), packed.data.data_ptr(),
                           packed.data.numel(), Y.data_ptr(), M, N, K, flags,
                           None if workspace is None else workspace.data_ptr(),
                           0 if workspace is None else workspace.numel(), handle), "fp8_gemm")
    if stream is not None:
        _used_on(stream, xq, xs, packed.data, Y, workspace)
    return Y


def fp8_grouped_gemm(xq: torch.Tensor, xs: torch.Tensor, packed: PackedFP8, offsets: torch.Tensor,
                     rows: Optional[torch.Tensor] = None, out: str = "bf16",
                     Y: Optional[torch.Tensor] = None, plan=None, stream=None) -> torch.Tensor:
    """Y [R][N]: rows offsets[e] .. offsets[e+1]-1 are rows of xq times the weights of expert e.
    offsets int32 [E+1] on the device (never read by the host); output row r is made from row
    rows[r] of xq (int32 [R]), or from row r if rows is None (then R = xq.shape[0])."""
    where = "fp8_grouped_gemm"
    T, K, flag, tdt = _rows(where, xq, xs, packed, out)
    E, N = packed.E, packed.N
    _require(offsets, f"{where}: offsets", torch.int32, E + 1, xq.device)
    R = T
    if rows is not None:
        R = rows.numel()
        _require(rows, f"{where}: rows", torch.int32, R, xq.device)
    if Y is None:
        Y = (torch.empty((R, N), dtype=tdt, device=xq.device) if stream is None
             else _empty_on(stream, (R, N), tdt, xq.device))
    else:
        _require(Y, f"{where}: Y", tdt, R * N, xq.device)
    flags = flag if plan is None else flag | plan_flags_fp8(plan)
    _check(_lib().fp8_grouped_gemm(xq.data_ptr(), xs.data_ptr(), packed.data.data_ptr(),
                                   packed.data.numel(), offsets.data_ptr(),
                                   None if rows is None else rows.data_ptr(), Y.data_ptr(), R, T,
                                   E, N, K, flags, _stream_handle(stream)), where)
    if stream is not None:
        _used_on(stream, xq, xs, packed.data, offsets, rows, Y)
    return Y
