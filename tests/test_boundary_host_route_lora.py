"""The entry points of include/route.h and include/lora.h and their Python binding on the
host: exported, sized, and rejecting bad arguments before any HIP call (no call here passes
validation, or it has no work)."""
import ctypes
import os
import re

import pytest
import torch

import w4a16_dequant_gemm_amd as w4
from w4a16_dequant_gemm_amd import build as hipbuild

from host_fakes import FakeLibrary, FakeTensor, fake

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)
INV, UNS, OK, WS = (w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_UNSUPPORTED, w4.W4A16_OK,
                    w4.W4A16_ERR_WORKSPACE)
F16, BF16, F32, I32, U8 = (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.uint8)


def at(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hipbuild.LIB):
        hipbuild.build()
    from w4a16_dequant_gemm_amd import lora, route
    route._lib()
    lora._lib()
    return w4.load_library()


@pytest.mark.parametrize("header", ["route", "lora"])
def test_exports_every_declared_symbol(lib, header):
    from w4a16_dequant_gemm_amd import lora, route
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header + ".h")).read(),
                  flags=re.S)
    names = sorted(set(re.findall(r"\b(%s_[a-z0-9_]+)\s*\(" % header, text)))
    for name in names:
        assert hasattr(lib, name)
    known = {"route": route.C_FUNCTIONS_ROUTE, "lora": lora.C_FUNCTIONS_LORA}[header]
    assert sorted(known) == names


def test_route_tokens_rejects_before_any_launch(lib):
    def call(l=FAKE, ld=64, v=None, w=FAKE, e=FAKE, c=FAKE, o=FAKE, r=FAKE, p=FAKE, loss=None,
             pull=None, T=100, E=64, top=8, flags=2, ws=None, wb=0):
        return lib.route_tokens(l, ld, v, w, e, c, o, r, p, loss, pull, T, E, top, flags, ws, wb,
                                None)
    assert call() == WS                       # the last check of all
    assert call(ws=FAKE, wb=100) == WS
    assert call(ws=at(8), wb=1 << 30) == INV
    assert call(flags=3) == INV
    assert call(flags=4) == INV
    assert call(flags=0x20) == INV
    assert call(T=-1) == INV
    assert call(T=1 << 26) == INV
    assert call(T=1 << 25, E=1024, ld=1024, top=32) == WS     # 2^30 slots
    assert call(E=0) == INV
    assert call(E=1025, ld=1025) == UNS
    assert call(top=0) == INV
    assert call(top=65) == INV
    assert call(top=33) == UNS
    assert call(ld=63) == INV
    assert call(ld=1 << 40) == INV
    assert call(l=None) == INV
    assert call(l=at(2)) == INV
    assert call(l=at(2), flags=1) == WS
    assert call(l=at(1), flags=1) == INV
    for bad in (None, at(2)):
        for name in "wecorp":
            assert call(**{name: bad}) == INV, name
    assert call(loss=FAKE) == INV             # the loss without its slopes
    assert call(pull=FAKE) == INV
    assert call(loss=at(2), pull=FAKE) == INV
    assert call(T=0) == WS                    # writes zeros like any other call
    assert call(T=0, l=None, w=None, e=None, r=None, p=None) == WS


def test_route_workspace(lib):
    size = lib.route_workspace_bytes
    assert size(64, 1024, 32) == 0            # one workgroup does all of it
    assert size(1, 1, 1) == 0
    assert size(65, 64, 8) > 65536
    assert size(0, 64, 8) > 65536
    for bad in ((-1, 64, 8), (100, 0, 1), (100, 2000, 8), (100, 8, 9), (1 << 26, 8, 8)):
        assert size(*bad) == 0
    # a small part of the logits
    assert size(1 << 20, 256, 8) < (1 << 20) * 256 // 4


def test_route_backward_rejects_before_any_launch(lib):
    def call(l=FAKE, ld=64, v=None, w=FAKE, e=FAKE, pull=FAKE, dw=FAKE, dl=FAKE, out=FAKE, T=4,
             E=64, top=8, flags=2):
        return lib.route_tokens_backward(l, ld, v, w, e, pull, dw, dl, out, T, E, top, flags, None)
    assert call(T=0) == OK
    assert call(T=0, l=None, w=None, e=None, out=None) == OK
    assert call(pull=None) == INV             # a loss's gradient without its slopes
    assert call(T=0, pull=None) == INV
    for name in ("l", "w", "e", "out"):
        assert call(**{name: None}) == INV
        assert call(**{name: at(2)}) == INV
    for name in ("dw", "dl", "pull"):
        assert call(**{name: at(2)}) == INV
    assert call(ld=10) == INV
    assert call(flags=7) == INV
    assert call(top=65) == INV
    assert call(E=2000, ld=2000) == UNS


def test_combine_rejects_before_any_launch(lib):
    def call(y=FAKE, ldy=256, w=FAKE, p=FAKE, r=None, ldr=0, out=FAKE, T=4, R=8, N=256, top=2,
             flags=1):
        return lib.route_combine(y, ldy, w, p, r, ldr, out, T, R, N, top, flags, None)
    assert call(T=0) == OK
    assert call(flags=2) == INV               # rows are 16-bit
    assert call(ldy=255) == INV
    assert call(r=FAKE, ldr=255) == INV
    assert call(N=0) == INV
    assert call(N=1 << 24, ldy=1 << 24) == INV
    assert call(R=-1) == INV
    assert call(top=0) == INV
    assert call(top=33) == UNS
    assert call(T=1 << 26) == INV
    for name in ("y", "w", "p", "out"):
        assert call(**{name: None}) == INV
        assert call(**{name: at(1)}) == INV
    assert call(r=at(1), ldr=256) == INV

    def back(d=FAKE, ldd=256, y=FAKE, ldy=256, w=FAKE, p=FAKE, n=FAKE, dy=FAKE, dw=FAKE, T=4, R=8,
             N=256, top=2, flags=1):
        return lib.route_combine_backward(d, ldd, y, ldy, w, p, n, dy, dw, T, R, N, top, flags,
                                          None)
    assert back(T=0, R=0) == OK
    assert back(R=9) == INV                   # rows that no token would clear
    assert back(ldd=10) == INV
    assert back(flags=2) == INV
    for name in ("d", "y", "w", "p", "dy", "dw"):
        assert back(**{name: None}) == INV
        assert back(**{name: at(1)}) == INV
    assert back(n=at(2)) == INV


def test_lora_rejects_before_any_launch(lib):
    def call(base=FAKE, ldb=256, x=FAKE, ldx=512, xs=None, a=FAKE, b=FAKE, s=None, ids=FAKE,
             out=at(1 << 20), ldo=256, M=4, N=256, K=512, R=16, L=3, flags=0, ws=None, wb=0):
        return lib.lora_add(base, ldb, x, ldx, xs, a, b, s, ids, out, ldo, M, N, K, R, L, flags,
                            ws, wb, None)
    assert call() == WS                       # the last check of all
    assert call(ws=FAKE, wb=65536) == WS
    assert call(ws=at(8), wb=1 << 30) == INV
    assert call(M=0) == OK
    assert call(M=-1) == INV
    assert call(M=1 << 24) == INV
    assert call(M=(1 << 24) - 1, N=1 << 14, ldb=1 << 14, ldo=1 << 14) == INV    # 2^38 outputs
    assert call(N=0) == INV
    assert call(K=516, ldx=520) == UNS
    assert call(K=520, ldx=520) == WS
    assert call(K=520, ldx=528, flags=0x10, xs=FAKE) == UNS
    assert call(R=12) == UNS
    assert call(R=264) == UNS
    assert call(R=0) == INV
    assert call(L=0) == INV
    assert call(flags=2) == INV
    assert call(flags=0x20) == INV
    assert call(flags=0x10) == INV            # codes without scales
    assert call(xs=FAKE) == INV               # scales without codes
    assert call(flags=0x10, xs=at(2)) == INV
    assert call(ldx=504) == INV
    assert call(ldx=516) == INV
    assert call(ldx=520, flags=0x10, xs=FAKE) == INV
    assert call(ldb=255) == INV
    assert call(ldo=255) == INV
    assert call(out=FAKE, ldo=264) == INV     # in place with another stride
    for name in ("base", "x", "a", "b", "ids", "out"):
        assert call(**{name: None}) == INV
    for name in ("x", "a", "b"):
        assert call(**{name: at(8)}) == INV
    for name in ("base", "out"):
        assert call(**{name: at(1)}) == INV
        assert call(**{name: at((1 << 20) + 2)}) == WS
    assert call(s=at(2)) == INV
    assert call(ids=at(2)) == INV


def test_lora_workspace(lib):
    size = lib.lora_workspace_bytes
    assert size(0, 256, 512, 16, 4, 0) == 0
    assert size(4, 256, 512, 12, 4, 0) == 0
    assert size(4, 256, 512, 16, 4, 0x40) == 0
    assert size(4, 256, 512, 16, 0, 0) == 0
    for M, N, K, R, L in ((1, 1, 8, 8, 1), (64, 28672, 8192, 16, 32), (4096, 28672, 8192, 64, 4),
                          (300, 64, 512, 16, 64), (300, 64, 512, 16, 65),
                          (100000, 64, 28672, 256, 1000)):
        need = size(M, N, K, R, L, 0)
        places = M + 64 * (min(L, 64) + 1)     # adapters' rows begin whole groups
        # parts of the first product, and for many rows operands and an order
        assert 65536 + M * R * 4 <= need <= 65536 + places * (R * 64 + (R + 31) // 32 * 128 + 12)
        assert size(M, N, K, R, L, 1) == need


def test_binding_rejects_host_tensors(lib):
    from w4a16_dequant_gemm_amd import lora, route
    x = torch.zeros(2, 256, dtype=BF16)
    with pytest.raises(w4.W4A16Error):
        route.route_tokens(x, 4)
    with pytest.raises(w4.W4A16Error):
        route.combine_rows(x, torch.zeros(1, 2), torch.zeros(1, 2, dtype=I32))
    with pytest.raises(w4.W4A16Error):
        lora.lora_add(x, x, torch.zeros(1, 8, 256, dtype=BF16), torch.zeros(1, 256, 8, dtype=BF16),
                      torch.zeros(2, dtype=I32))


# ---- what the binding checks of its tensors, on stand-ins for them

class Strided(FakeTensor):
    def __init__(self, *shape, dtype, strides=None, index=0):
        super().__init__(*shape, dtype=dtype)
        self.strides, self.index = strides, index
        self.device = torch.device("cuda", index)

    def stride(self, i):
        return self.strides[i] if self.strides else super().stride(i)

    def is_contiguous(self):
        return self.strides is None

    def get_device(self):
        return self.index

    def element_size(self):
        return 1


class Buffer(FakeTensor):
    """One allocation that several outputs are parts of."""

    def as_strided(self, shape, strides, first):
        assert strides == (1,) or strides == (shape[1], 1)
        assert first + torch.Size(shape).numel() <= self.numel()
        return Buffer(*shape, dtype=self.dtype)

    def view(self, dtype):
        return Buffer(*self.shape, dtype=dtype)


@pytest.fixture
def bound(monkeypatch):
    from w4a16_dequant_gemm_amd import lora, route
    monkeypatch.setattr(w4, "_lib", FakeLibrary())
    for module in (route, lora):
        monkeypatch.setattr(module, "_lib", FakeLibrary)
        monkeypatch.setattr(module, "_ws_bytes", {})
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(w4, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None:
                        Buffer(*((shape,) if isinstance(shape, int) else shape), dtype=dtype))
    monkeypatch.setattr(torch, "empty_like", lambda like: FakeTensor(*like.shape, dtype=like.dtype))
    return route, lora


def refused(f, *args, **kw):
    with pytest.raises(w4.W4A16Error):
        f(*args, **kw)


def test_route_tokens_checks(bound):
    route, _ = bound
    logits = fake(6, 16, dtype=F32)
    r = route.route_tokens(logits, 4, balance=True)
    assert r.experts.shape == (6, 4) and r.offsets.shape == (17,) and r.loss.shape == ()
    assert route.route_tokens(logits, 4).loss is None
    route.route_tokens(Strided(6, 16, dtype=BF16, strides=(40, 1)), 4)
    refused(route.route_tokens, Strided(6, 16, dtype=F32, strides=(1, 6)), 4)
    refused(route.route_tokens, Strided(6, 16, dtype=F32, strides=(8, 1)), 4)
    refused(route.route_tokens, fake(6, 16, dtype=torch.float64), 4)
    refused(route.route_tokens, fake(2, 3, 16, dtype=F32), 4)
    refused(route.route_tokens, logits, 0)
    refused(route.route_tokens, logits, 17)
    refused(route.route_tokens, logits, 4, valid=fake(5, dtype=torch.bool))
    refused(route.route_tokens, logits, 4, valid=fake(6, dtype=F32))
    route.route_tokens(logits, 4, valid=fake(6, dtype=torch.bool))
    refused(route.route_tokens, Strided(6, 16, dtype=F32, index=1), 4)   # not the current device
    refused(route.route_tokens, logits, 4, workspace=Strided(1 << 20, dtype=U8, index=1))

    back = route.route_tokens_backward
    assert back(logits, r, fake(6, 4, dtype=F32), fake(dtype=F32)).shape == (6, 16)
    refused(back, logits, r, fake(6, 3, dtype=F32))
    refused(back, logits, r, fake(6, 4, dtype=BF16))
    refused(back, fake(5, 16, dtype=F32), r)
    refused(back, logits, r, None, fake(2, dtype=F32))
    r.pull = None
    refused(back, logits, r, None, fake(dtype=F32))
    back(logits, r, fake(6, 4, dtype=F32))


def test_combine_checks(bound):
    route, _ = bound
    y, w, p = fake(12, 40, dtype=BF16), fake(6, 2, dtype=F32), fake(6, 2, dtype=I32)
    assert route.combine_rows(y, w, p).shape == (6, 40)
    res = fake(6, 40, dtype=BF16)
    assert route.combine_rows(y, w, p, residual=res, out=res) is res
    refused(route.combine_rows, fake(12, 40, dtype=F32), w, p)
    refused(route.combine_rows, y, fake(6, 2, dtype=BF16), p)
    refused(route.combine_rows, y, fake(5, 2, dtype=F32), p)
    refused(route.combine_rows, y, w, fake(6, 2, dtype=torch.int64))
    refused(route.combine_rows, y, w, p, residual=fake(6, 41, dtype=BF16))
    refused(route.combine_rows, y, w, p, residual=fake(6, 40, dtype=F16))
    refused(route.combine_rows, y, w, p, out=fake(5, 40, dtype=BF16))
    off = fake(5, dtype=I32)
    back = route.combine_rows_backward
    dy, dw = back(res, y, w, p, off)
    assert dy.shape == (12, 40) and dw.shape == (6, 2)
    refused(back, fake(6, 41, dtype=BF16), y, w, p, off)
    refused(back, res, fake(13, 40, dtype=BF16), w, p, off)
    refused(back, res, y, w, p, fake(5, dtype=torch.int64))
    refused(back, res, y, w, p, fake(0, dtype=I32))


def test_lora_checks(bound):
    _, lora = bound
    good = dict(base=fake(6, 40, dtype=BF16), x=fake(6, 64, dtype=BF16),
                a=fake(3, 8, 64, dtype=BF16), b=fake(3, 40, 8, dtype=BF16), ids=fake(6, dtype=I32))

    def call(**change):
        return lora.lora_add(**{**good, **change})
    assert call().shape == (6, 40)
    assert call(out=good["base"]) is good["base"]
    for change in (dict(x=fake(5, 64, dtype=BF16)), dict(x=fake(6, 64, dtype=F16)),
                   dict(x=fake(6, 64, dtype=U8)), dict(base=fake(6, 40, dtype=F32)),
                   dict(a=fake(3, 8, 72, dtype=BF16)), dict(a=fake(2, 8, 64, dtype=BF16)),
                   dict(b=fake(3, 41, 8, dtype=BF16)), dict(b=fake(3, 40, 8, dtype=F16)),
                   dict(b=Strided(3, 40, 8, dtype=BF16, strides=(320, 1, 40))),
                   dict(ids=fake(6, dtype=torch.int64)), dict(ids=fake(7, dtype=I32)),
                   dict(scale=fake(6, dtype=F32)), dict(scale=fake(3, dtype=BF16)),
                   dict(out=fake(6, 41, dtype=BF16)), dict(out=fake(6, 40, dtype=F16)),
                   dict(base=Strided(6, 40, dtype=BF16, strides=(8, 1))),
                   dict(xs=fake(6, 1, dtype=F32)),
                   dict(x=fake(6, 64, dtype=U8), xs=fake(6, 2, dtype=F32)),
                   dict(x=Strided(6, 64, dtype=BF16, index=1))):
        refused(call, **change)
    call(x=fake(6, 64, dtype=U8), xs=fake(6, 1, dtype=F32))
    refused(call, x=fake(6, 256, dtype=U8), a=fake(3, 8, 256, dtype=BF16),
            xs=fake(2, 6, dtype=F32))                                  # laid out by block


def test_captured_calls_have_scratch_of_their_own(monkeypatch):
    made = []
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True)
    monkeypatch.setattr(w4, "_empty_on", lambda *args: made.append(args) or "own")
    monkeypatch.setattr(w4, "_workspace_at", lambda *args: "shared")
    device = torch.device("cuda", 0)
    assert w4._scratch(100, device, None, 7) == "own"
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)
    assert w4._scratch(100, device, None, 7) == "shared"
    monkeypatch.setattr(w4, "_capture_number", lambda handle: 3 if handle == 9 else None)
    assert w4._scratch(100, device, "s", 9) == "own"
    assert w4._scratch(100, device, "s", 7) == "shared"
    assert len(made) == 2
