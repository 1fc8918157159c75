"""What the fp8 and row-quantiser bindings check of their tensors before the library is
called, on stand-ins for device tensors (no GPU)."""
import os
import re

import pytest
import torch

import w4a16_dequant_gemm_amd as w4
from w4a16_dequant_gemm_amd import fp8, rowquant

from host_fakes import FakeLibrary, FakeTensor, fake

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, U8, I32 = torch.float32, torch.uint8, torch.int32


@pytest.fixture(autouse=True)
def _library(monkeypatch):
    monkeypatch.setattr(w4, "_lib", FakeLibrary())
    monkeypatch.setattr(w4, "_stream_handle", lambda stream: 0)
    for module in (fp8, rowquant):
        monkeypatch.setattr(module, "_lib", FakeLibrary)
        monkeypatch.setattr(module, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(fp8, "_ws_bytes", {})
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None:
                        FakeTensor(*((shape,) if isinstance(shape, int) else shape), dtype=dtype))
    monkeypatch.setattr(torch, "empty_like", lambda like, dtype=None:
                        FakeTensor(*like.shape, dtype=dtype or like.dtype))


def blob(grouped=False, K=512):
    return fp8.PackedFP8(fake(1 << 20, dtype=U8), 1, K, 128, grouped)


@pytest.mark.parametrize("grouped", [False, True])
def test_scales_laid_out_by_block_are_refused(grouped):
    """[K/128][rows] has as many numbers as [rows][K/128] and means another product."""
    def call(xs):
        xq = fake(6, 512, dtype=U8)
        if grouped:
            return fp8.fp8_grouped_gemm(xq, xs, blob(True), fake(2, dtype=I32))
        return fp8.fp8_gemm(xq, xs, blob())
    assert call(fake(6, 4, dtype=F32)).shape == (6, 128)
    assert call(fake(24, dtype=F32)).shape == (6, 128)          # flat, in that order
    assert call(fake(2, 3, 4, dtype=F32)).shape == (6, 128)
    for shape in ((4, 6), (24, 1), (1, 24), (2, 12)):
        with pytest.raises(w4.W4A16Error):
            call(fake(*shape, dtype=F32))


@pytest.mark.parametrize("kind,dtype,n", [("fp8", F32, 5), ("mx", U8, 20)])
def test_scale_outputs_laid_out_by_block_are_refused(kind, dtype, n):
    x, w = fake(6, 640, dtype=torch.float16), fake(640, dtype=torch.float16)
    calls = (lambda s: rowquant.rmsnorm_quantize_rows(x, w, kind=kind, s=s),
             lambda s: rowquant.swiglu_quantize_rows(x, x, kind=kind, s=s))
    for call in calls:
        for shape in ((6, n), (6 * n,), (2, 3, n)):
            given = fake(*shape, dtype=dtype)
            assert call(given)[1] is given
        for shape in ((n, 6), (6 * n, 1)):
            with pytest.raises(w4.W4A16Error):
                call(fake(*shape, dtype=dtype))


class Elsewhere(FakeTensor):
    """A tensor in host memory, or on another device, or with gaps."""

    def __init__(self, cuda=True, index=0, contiguous=True):
        super().__init__(1 << 20, dtype=U8)
        self.is_cuda, self.index, self.contiguous = cuda, index, contiguous

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous


def test_a_workspace_the_kernel_cannot_use_is_refused():
    """Its address and element count go to the library as they are."""
    half = torch.float16
    p16 = w4.PackedW4(fake(1 << 20, dtype=U8), 512, 128, 128, 0, w4._layout_version)
    calls = (lambda ws: fp8.fp8_gemm(fake(6, 512, dtype=U8), fake(6, 4, dtype=F32), blob(),
                                     workspace=ws),
             lambda ws: w4.w4a16_gemm(fake(6, 512, dtype=half), p16, workspace=ws),
             lambda ws: w4.w4a16_gemm_ex(fake(6, 512, dtype=half), p16, workspace=ws))
    for call in calls:
        assert call(Elsewhere()).shape == (6, 128)
        for bad in (Elsewhere(cuda=False, index=-1), Elsewhere(index=1),
                    Elsewhere(contiguous=False)):
            with pytest.raises(w4.W4A16Error):
                call(bad)


def test_a_blob_of_another_layout_is_refused():
    """One kept from a library that ordered the weights otherwise."""
    header = open(os.path.join(ROOT, "include", "fp8.h")).read()
    assert int(re.search(r"#define FP8_LAYOUT_VERSION (\d+)", header)[1]) == fp8.FP8_LAYOUT_VERSION
    xq, xs = fake(6, 512, dtype=U8), fake(6, 4, dtype=F32)
    for grouped, call in ((False, lambda p: fp8.fp8_gemm(xq, xs, p)),
                          (True, lambda p: fp8.fp8_grouped_gemm(xq, xs, p, fake(2, dtype=I32)))):
        packed = blob(grouped)
        assert call(packed).shape == (6, 128)
        packed.layout_version = fp8.FP8_LAYOUT_VERSION + 1
        with pytest.raises(w4.W4A16Error):
            call(packed)


def test_workspace_sizes_are_kept_by_device_and_not_forever(monkeypatch):
    asked = []

    def need(M, N, K, *rest):
        asked.append(M)
        return 64 * M
    monkeypatch.setattr(fp8, "fp8_workspace_bytes", need)
    monkeypatch.setattr(w4, "w4a16_workspace_bytes", need)
    monkeypatch.setattr(w4, "_ws_bytes", {})
    for kept, ask in ((fp8._ws_bytes, lambda d, m: fp8._workspace_need(d, m, 128, 512, 0)),
                      (w4._ws_bytes, lambda d, m: w4._workspace_need(d, m, 128, 512, 128, 0))):
        asked.clear()
        assert [ask(0, 5), ask(0, 5), ask(1, 5), ask(0, 5)] == [320] * 4
        assert asked == [5, 5]                      # once per device
        for m in range(20000):
            assert ask(0, m) == 64 * m
        assert len(kept) <= 4096
