"""Python binding of what stands round the product grouped by expert (include/route.h) of
libw4a16.so: the router with its balance loss, the weighted sum of the experts' rows, and
their gradients.

    r = route_tokens(logits, top)                      offsets and rows for
    y = fp8.fp8_grouped_gemm(q, s, packed, r.offsets, rows=r.rows)
    out = combine_rows(y, r.weights, r.places, residual=h)

None of the calls is part of torch's autograd graph: what they return has no grad_fn, whether or
not an argument requires a gradient.  A training program calls the *_backward functions itself,
for instance from a torch.autograd.Function.  The products between the router and the sum
have no backward here: dy is where the program's own begins.

Argument marshalling only; there is no fallback.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import (_bad, _check, _empty_on, _keep_bytes, _launch_stream, _require,
               _require_workspace, _scratch, _used_on, load_library)

C_FUNCTIONS_ROUTE = ("route_workspace_bytes", "route_tokens", "route_tokens_backward",
                     "route_combine", "route_combine_backward")
_TYPES = {torch.float16: 0x0, torch.bfloat16: 0x1, torch.float32: 0x2}
_ROW_TYPES = (torch.float16, torch.bfloat16)
_RENORMALIZE = 0x10

_declared = None
_ws_bytes = {}


def _lib():
    global _declared
    if _declared is None:
        lib = load_library()
        p, i64, u32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
        lib.route_workspace_bytes.argtypes = [i64, i64, i64]
        lib.route_workspace_bytes.restype = sz
        lib.route_tokens.argtypes = [p, i64, p, p, p, p, p, p, p, p, p, i64, i64, i64, u32, p, sz, p]
        lib.route_tokens.restype = ctypes.c_int
        lib.route_tokens_backward.argtypes = [p, i64, p, p, p, p, p, p, p, i64, i64, i64, u32, p]
        lib.route_tokens_backward.restype = ctypes.c_int
        lib.route_combine.argtypes = [p, i64, p, p, p, i64, p, i64, i64, i64, i64, u32, p]
        lib.route_combine.restype = ctypes.c_int
        lib.route_combine_backward.argtypes = [p, i64, p, i64, p, p, p, p, p, i64, i64, i64, i64,
                                               u32, p]
        lib.route_combine_backward.restype = ctypes.c_int
        _declared = lib
    return _declared


@dataclass
class Routing:
    """What route_tokens decided for T tokens, top slots each, over E experts."""
    weights: torch.Tensor            # float32 [T][top]
    experts: torch.Tensor            # int32 [T][top], -1: the slot has no expert
    counts: torch.Tensor             # int32 [E], slots of each expert
    offsets: torch.Tensor            # int32 [E+1], rows of each expert
    rows: torch.Tensor               # int32 [T*top], the token of each row, -1 behind the last
    places: torch.Tensor             # int32 [T][top], the row of each slot, -1: none
    loss: Optional[torch.Tensor]     # float32 [], the balance loss
    pull: Optional[torch.Tensor]     # float32 [E], the loss's slope by each sum of p
    renormalize: bool
    valid: Optional[torch.Tensor]


def route_workspace_bytes(T: int, E: int, top: int) -> int:
    return int(_lib().route_workspace_bytes(T, E, top))


def _rows(t: torch.Tensor, where: str, name: str, dtypes) -> int:
    """Checks a [rows][W] tensor; returns the rows' distance in elements."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        _bad(f"{where}: {name}: need a [rows][columns] device tensor of "
             f"{[str(d) for d in dtypes]}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    n, W = t.shape
    ld = t.stride(0) if n > 1 else W   # the stride of a single row is never used
    if (t.stride(1) != 1 and W > 1) or ld < W:
        _bad(f"{where}: {name}: rows must be contiguous and not overlap")
    return ld


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """An output of t's shape and dtype, contiguous."""
    # empty_like: 1.2 us where empty with a shape and a device takes 1.7
    return (torch.empty_like(t) if stream is None and t.is_contiguous()
            else _empty_on(stream, tuple(t.shape), t.dtype, t.device))


def _valid_pointer(valid, where: str, T: int, device):
    if valid is None:
        return None
    if valid.dtype != torch.bool and valid.dtype != torch.uint8:
        _bad(f"{where}: valid must be bool or uint8")
    _require(valid, f"{where}: valid", valid.dtype, T, device)
    return valid.data_ptr()


def route_tokens(logits: torch.Tensor, top: int, renormalize: bool = True,
                 valid: Optional[torch.Tensor] = None, balance: bool = False,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> Routing:
    """The experts of every token: the top largest of softmax(logits [T][E]) (fp32, fp16 or
    bf16, rows may be strided), equal ones by the lowest index, with their weights (divided
    by their sum if renormalize), counts and order; with balance also the balance loss.
    valid (bool or uint8 [T]) is 0 for tokens of padding, which get no expert."""
    where = "route_tokens"
    ld = _rows(logits, where, "logits", _TYPES)
    T, E = logits.shape
    top = int(top)
    if top < 1 or top > E:
        _bad(f"{where}: top is {top}, there are {E} experts")
    dev, device = logits.get_device(), logits.device
    v = _valid_pointer(valid, where, T, device)
    # one allocation for the outputs: offsets and rows, which the products read, 16-byte
    # aligned (6 allocations take 10 us, one and its parts 7)
    n, at_rows = T * top, (E + 4) // 4 * 4
    whole = _empty_on(stream, (at_rows + 4 * n + E,), torch.int32, device)
    shape, strides = (T, top), (top, 1)
    offsets = whole.as_strided((E + 1,), (1,), 0)
    rows = whole.as_strided((n,), (1,), at_rows)
    experts = whole.as_strided(shape, strides, at_rows + n)
    places = whole.as_strided(shape, strides, at_rows + 2 * n)
    weights = whole.as_strided(shape, strides, at_rows + 3 * n).view(torch.float32)
    counts = whole.as_strided((E,), (1,), at_rows + 4 * n)
    loss = _empty_on(stream, (), torch.float32, device) if balance else None
    pull = _empty_on(stream, (E,), torch.float32, device) if balance else None
    handle = _launch_stream(where, stream, dev)
    if workspace is None:
        key = (T, E, top)
        need = _ws_bytes.get(key)
        if need is None:
            need = _keep_bytes(_ws_bytes, key, route_workspace_bytes(T, E, top))
        if need:
            workspace = _scratch(need, logits.device, stream, handle)
    else:
        _require_workspace(workspace, where, dev)
    flags = _TYPES[logits.dtype] | (_RENORMALIZE if renormalize else 0)
    _check(_lib().route_tokens(logits.data_ptr(), ld, v, weights.data_ptr(), experts.data_ptr(),
                               counts.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
                               places.data_ptr(), loss.data_ptr() if balance else None,
                               pull.data_ptr() if balance else None, T, E, top, flags,
                               None if workspace is None else workspace.data_ptr(),
                               0 if workspace is None
                               else workspace.numel() * workspace.element_size(), handle), where)
    if stream is not None:
        _used_on(stream, logits, valid, workspace)
    return Routing(weights, experts, counts, offsets, rows, places, loss, pull, bool(renormalize),
                   valid)


def route_tokens_backward(logits: torch.Tensor, routing: Routing,
                          dweights: Optional[torch.Tensor] = None,
                          dloss: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dlogits [T][E] in the logits' dtype: the gradient of routing.weights by dweights (float32
    [T][top]) and of routing.loss by dloss (float32, one element on the device)."""
    where = "route_tokens_backward"
    ld = _rows(logits, where, "logits", _TYPES)
    T, E = logits.shape
    device = logits.device
    top = routing.weights.shape[-1]
    v = _valid_pointer(routing.valid, where, T, device)
    _require(routing.weights, f"{where}: weights", torch.float32, T * top, device)
    _require(routing.experts, f"{where}: experts", torch.int32, T * top, device)
    if dweights is not None:
        _require(dweights, f"{where}: dweights", torch.float32, T * top, device)
    if dloss is not None:
        _require(dloss, f"{where}: dloss", torch.float32, 1, device)
        _require(routing.pull, f"{where}: pull (of a call with balance)", torch.float32, E, device)
    dlogits = _like(logits, stream)
    flags = _TYPES[logits.dtype] | (_RENORMALIZE if routing.renormalize else 0)
    _check(_lib().route_tokens_backward(
        logits.data_ptr(), ld, v, routing.weights.data_ptr(), routing.experts.data_ptr(),
        None if routing.pull is None else routing.pull.data_ptr(),
        None if dweights is None else dweights.data_ptr(),
        None if dloss is None else dloss.data_ptr(), dlogits.data_ptr(), T, E, top, flags,
        _launch_stream(where, stream, logits.get_device())), where)
    if stream is not None:
        _used_on(stream, logits, routing.valid, routing.weights, routing.experts, routing.pull,
                 dweights, dloss)
    return dlogits


def _slots(weights: torch.Tensor, places: torch.Tensor, where: str, T: int, device) -> int:
    if weights.dim() != 2 or weights.shape[0] != T:
        _bad(f"{where}: weights is {tuple(weights.shape)}, there are {T} tokens")
    top = weights.shape[1]
    _require(weights, f"{where}: weights", torch.float32, T * top, device)
    _require(places, f"{where}: places", torch.int32, T * top, device)
    return top


def combine_rows(y: torch.Tensor, weights: torch.Tensor, places: torch.Tensor,
                 residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """out [T][N] = residual + the sum over slots of weights [T][top] times the rows of y [R][N]
    (fp16 or bf16, rows may be strided) that places [T][top] name; a place outside [0, R) adds
    nothing.  out, if given, is the contiguous tensor to write (residual itself, or one that
    overlaps no input)."""
    where = "combine_rows"
    ldy = _rows(y, where, "y", _ROW_TYPES)
    R, N = y.shape
    T, device = places.shape[0], y.device
    top = _slots(weights, places, where, T, device)
    ldr = N
    if residual is not None:
        ldr = _rows(residual, where, "residual", (y.dtype,))
        if tuple(residual.shape) != (T, N) or residual.get_device() != y.get_device():
            _bad(f"{where}: residual is {tuple(residual.shape)} on {residual.device}")
    if out is None:
        out = (_like(residual, stream) if residual is not None
               else _empty_on(stream, (T, N), y.dtype, device))
    else:
        _require(out, f"{where}: out", y.dtype, T * N, device)
    _check(_lib().route_combine(y.data_ptr(), ldy, weights.data_ptr(), places.data_ptr(),
                                None if residual is None else residual.data_ptr(), ldr,
                                out.data_ptr(), T, R, N, top, _TYPES[y.dtype],
                                _launch_stream(where, stream, y.get_device())), where)
    if stream is not None:
        _used_on(stream, y, weights, places, residual, out)
    return out


def combine_rows_backward(dout: torch.Tensor, y: torch.Tensor, weights: torch.Tensor,
                          places: torch.Tensor, offsets: torch.Tensor, stream=None):
    """(dy [R][N], dweights [T][top]) of combine_rows: dy[places] = weights * dout rounded to
    y's dtype, zeros from row offsets[-1] on; dweights float32, 0 for a place outside
    [0, R).  offsets as route_tokens gave them (every row before the last of them has its
    slot), R = T * top at most."""
    where = "combine_rows_backward"
    ldy = _rows(y, where, "y", _ROW_TYPES)
    ldd = _rows(dout, where, "dout", (y.dtype,))
    R, N = y.shape
    T, device = places.shape[0], y.device
    if tuple(dout.shape) != (T, N) or dout.get_device() != y.get_device():
        _bad(f"{where}: dout is {tuple(dout.shape)} on {dout.device}, y {tuple(y.shape)}")
    top = _slots(weights, places, where, T, device)
    _require(offsets, f"{where}: offsets", torch.int32, offsets.numel(), device)
    if offsets.numel() < 1 or R > T * top:
        _bad(f"{where}: {R} rows for {T} tokens of {top} slots, {offsets.numel()} offsets")
    dy, dweights = _like(y, stream), _like(weights, stream)
    _check(_lib().route_combine_backward(dout.data_ptr(), ldd, y.data_ptr(), ldy,
                                         weights.data_ptr(), places.data_ptr(),
                                         offsets.data_ptr() + 4 * (offsets.numel() - 1),
                                         dy.data_ptr(), dweights.data_ptr(), T, R, N, top,
                                         _TYPES[y.dtype],
                                         _launch_stream(where, stream, y.get_device())), where)
    if stream is not None:
        _used_on(stream, dout, y, weights, places, offsets)
    return dy, dweights
