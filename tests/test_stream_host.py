"""Streams in the Python binding, without a GPU: torch's stream functions are replaced by
ones that only note which stream is current when memory is made."""
import contextlib

import pytest
import torch

import w4a16_dequant_gemm_amd as w4

from host_fakes import FakeLibrary, FakeTensor, fake

CURRENT = 0x10


class Streams:
    """Stands in for torch's current stream: a stack of handles."""

    def __init__(self, monkeypatch):
        self.stack, self.made = [CURRENT], []
        monkeypatch.setattr(torch.cuda, "ExternalStream",
                            lambda handle, device=None: ("external", handle, device))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", 0, device))
        monkeypatch.setattr(torch.cuda, "stream", self.use)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stack[-1])
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: self.stack[-1])
        zeros = torch.zeros

        def noted(*shape, dtype=None, device=None):
            self.made.append(("zeros", self.stack[-1]))
            return zeros(*shape, dtype=dtype)
        monkeypatch.setattr(torch, "zeros", noted)
        monkeypatch.setattr(w4, "_workspaces", {})
        monkeypatch.setattr(w4, "_retired_workspaces", [])
        monkeypatch.setattr(w4, "_captured_workspaces", {}, raising=False)
        self.capture = None
        monkeypatch.setattr(w4, "_capture_number", lambda handle: self.capture, raising=False)

    @contextlib.contextmanager
    def use(self, stream):
        self.stack.append(stream[1])
        yield
        self.stack.pop()


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


@pytest.mark.parametrize("handle", [CURRENT, 0x20, 0])
def test_workspace_is_filled_on_the_stream_that_uses_it(streams, handle):
    ws = w4._workspace_at(1 << 20, 0, handle)
    assert streams.made == [("zeros", handle)]
    assert w4._workspace_at(1 << 20, 0, handle) is ws
    w4._workspace_at((1 << 20) + 1, 0, handle)        # grows
    assert streams.made == [("zeros", handle)] * 2


def test_workspace_made_in_a_capture_serves_that_capture_alone(streams):
    """Its fill runs when that graph does: another graph, or a call outside, that found it
    would read counters no one has cleared."""
    streams.capture = 7
    first = w4._workspace_at(1 << 20, 0, 0x20)
    assert w4._workspace_at(1 << 10, 0, 0x20) is first
    streams.capture = 8
    second = w4._workspace_at(1 << 20, 0, 0x20)
    assert second is not first
    streams.capture = None
    outside = w4._workspace_at(1 << 20, 0, 0x20)
    assert outside is not first and outside is not second
    assert streams.made == [("zeros", 0x20)] * 3
    # one made and filled outside serves captures too, until they need a larger one
    streams.capture = 9
    assert w4._workspace_at(1 << 20, 0, 0x20) is outside
    larger = w4._workspace_at(1 << 21, 0, 0x20)
    assert larger.numel() == 1 << 21 and w4._workspace_at(1 << 21, 0, 0x20) is larger
    streams.capture = None
    assert w4._workspace_at(1 << 20, 0, 0x20) is outside


def calls(fake=fake):
    """name -> (a call with `stream=`, how many outputs it makes)."""
    from w4a16_dequant_gemm_amd import fp8, mxfp4, rowquant, w4a8
    half, u8, f32, i8, i32 = (torch.float16, torch.uint8, torch.float32, torch.int8, torch.int32)
    x, w = fake(4, 512, dtype=half), fake(512, dtype=half)
    rows = fake(4, 512, dtype=u8)
    blob = fake(1 << 20, dtype=u8)
    p16 = w4.PackedW4(blob, 512, 128, 128, 0, w4._layout_version)
    p8 = w4a8.PackedW8(blob, 512, 128, 128)
    one, many = (fp8.PackedFP8(blob, 1, 512, 128, g) for g in (False, True))
    xs, off = fake(4, 4, dtype=f32), fake(2, dtype=i32)
    return {
        "norm": (lambda s: rowquant.rmsnorm_quantize_rows(x, w, residual=x, stream=s), 3),
        "swiglu": (lambda s: rowquant.swiglu_quantize_rows(x, x, stream=s), 2),
        "fp8_gemm": (lambda s: fp8.fp8_gemm(rows, xs, one, stream=s), 1),
        "fp8_grouped_gemm": (lambda s: fp8.fp8_grouped_gemm(rows, xs, many, off, stream=s), 1),
        "fp8_repack": (lambda s: fp8.fp8_repack(fake(128, 512, dtype=u8), fake(1, 4, dtype=f32),
                                                stream=s), 1),
        "w4a16_gemm": (lambda s: w4.w4a16_gemm(x, p16, stream=s), 1),
        "w4a16_gemm_ex": (lambda s: w4.w4a16_gemm_ex(x, p16, stream=s), 1),
        "w4a16_dequant": (lambda s: w4.w4a16_dequant(p16, stream=s), 1),
        "w4a16_unrepack": (lambda s: w4.w4a16_unrepack(p16, stream=s), 3),
        "w4a8_quantize_rows": (lambda s: w4a8.w4a8_quantize_rows(x, stream=s), 2),
        "w4a8_gemm": (lambda s: w4a8.w4a8_gemm(fake(4, 512, dtype=i8), fake(4, dtype=f32), p8,
                                               stream=s), 1),
        "w4a8_dequant": (lambda s: w4a8.w4a8_dequant(p8, stream=s), 1),
        "mxfp4_quantize_rows": (lambda s: mxfp4.mxfp4_quantize_rows(x, stream=s), 2),
        "mxfp4_gemm": (lambda s: mxfp4.mxfp4_gemm(rows, fake(4, 16, dtype=u8),
                                                  mxfp4.PackedMX(blob, 512, 128), stream=s), 1),
    }


def without_library(monkeypatch):
    from w4a16_dequant_gemm_amd import fp8, mxfp4, rowquant, w4a8
    monkeypatch.setattr(w4, "_lib", FakeLibrary())
    for module in (fp8, rowquant, w4a8, mxfp4):
        monkeypatch.setattr(module, "_lib", FakeLibrary)
    monkeypatch.setattr(fp8, "_ws_bytes", {})
    monkeypatch.setattr(w4, "_ws_bytes", {})


NAMES = ["norm", "swiglu", "fp8_gemm", "fp8_grouped_gemm", "fp8_repack", "w4a16_gemm",
         "w4a16_gemm_ex", "w4a16_dequant", "w4a16_unrepack", "w4a8_quantize_rows", "w4a8_gemm",
         "w4a8_dequant", "mxfp4_quantize_rows", "mxfp4_gemm"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("handle", [CURRENT, 0x20, 0])
def test_outputs_are_made_on_the_stream_of_the_call(streams, monkeypatch, name, handle):
    """... and wait for torch's current stream too when they are dropped."""
    call, outputs = calls()[name]
    made, recorded = [], []

    def empty(shape, dtype=None, device=None):
        made.append(streams.stack[-1])
        return FakeTensor(*((shape,) if isinstance(shape, int) else shape), dtype=dtype,
                          recorded=recorded)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda like, dtype=None:
                        empty(like.shape, dtype=dtype or like.dtype))
    without_library(monkeypatch)
    call(handle)
    assert made == [handle] * outputs
    assert recorded == ([] if handle == CURRENT else [CURRENT] * outputs)


class TorchStream:
    """Stands in for torch.cuda.Stream."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_a_call_wait_for_its_stream_when_they_are_dropped(streams, monkeypatch, name):
    """... but not for a raw handle, which its owner may have destroyed by then."""
    monkeypatch.setattr(torch.cuda, "Stream", TorchStream)
    without_library(monkeypatch)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None:
                        fake(*((shape,) if isinstance(shape, int) else shape), dtype=dtype))
    monkeypatch.setattr(torch, "empty_like", lambda like, dtype=None:
                        fake(*like.shape, dtype=dtype or like.dtype))
    given = []

    def kept(*shape, dtype):
        given.append(FakeTensor(*shape, dtype=dtype))
        return given[-1]
    side = TorchStream(0x20)
    call, _ = calls(kept)[name]
    call(side)
    used = [t for t in given if side in t.recorded]
    assert len(used) >= 1 and all(t.recorded.count(side) <= 2 for t in used)
    expect = {"norm": 2, "swiglu": 1, "fp8_gemm": 3, "fp8_grouped_gemm": 4, "fp8_repack": 2,
              "w4a16_gemm": 2, "w4a16_gemm_ex": 2, "w4a16_dequant": 1, "w4a16_unrepack": 1,
              "w4a8_quantize_rows": 1, "w4a8_gemm": 3, "w4a8_dequant": 1,
              "mxfp4_quantize_rows": 1, "mxfp4_gemm": 3}
    assert len(used) == expect[name]
    given.clear()
    call, _ = calls(kept)[name]
    call(0x20)
    assert not any(t.recorded for t in given)
