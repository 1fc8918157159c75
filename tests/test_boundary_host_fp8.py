"""The fp8 and row-quantiser entry points (include/fp8.h, include/rowquant.h) on the
host: exported, sized, and rejecting bad arguments before any HIP call (no call here
passes validation, or it has no work)."""
import ctypes
import os
import re

import pytest
import torch

import w4a16_dequant_gemm_amd as w4
from w4a16_dequant_gemm_amd import build as hipbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)
FAKE_MIS = ctypes.c_void_p(0x10008)
INV, UNS, OK = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_UNSUPPORTED, w4.W4A16_OK


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hipbuild.LIB):
        hipbuild.build()
    from w4a16_dequant_gemm_amd import fp8, rowquant
    fp8._lib()
    rowquant._lib()
    return w4.load_library()


@pytest.mark.parametrize("header,prefix", [("fp8.h", "fp8"), ("rowquant.h", "rowquant")])
def test_exports_every_declared_symbol(lib, header, prefix):
    from w4a16_dequant_gemm_amd import fp8, rowquant
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(),
                  flags=re.S)
    names = sorted(set(re.findall(r"\b(%s_[a-z0-9_]+)\s*\(" % prefix, text)))
    for name in names:
        assert hasattr(lib, name)
    known = fp8.C_FUNCTIONS_FP8 if prefix == "fp8" else rowquant.C_FUNCTIONS_ROWQUANT
    assert sorted(known) == names


@pytest.mark.parametrize("E,K,N,expect", [
    (1, 256, 128, 256 * 128 + 16 + 64),                  # 2 scales, rounded up to 16 bytes
    (3, 144, 130, 3 * 256 * 256 + 3 * 2 * 2 * 4 + 64),   # padded to whole blocks
    (1, 8192, 28672, 8192 * 28672 + 64 * 224 * 4 + 64),
    (1, 100, 128, 0), (0, 128, 128, 0), (1, 0, 128, 0), (1, 128, 0, 0), (1, 1 << 24, 128, 0),
    (65536, 128, 128, 0)])
def test_packed_bytes(lib, E, K, N, expect):
    from w4a16_dequant_gemm_amd import fp8
    assert fp8.fp8_packed_bytes(E, K, N) == expect


def test_fp8_rejects_before_any_launch(lib):
    def gemm(xq=FAKE, xs=FAKE, p=FAKE, pb=1 << 40, Y=FAKE, M=4, N=256, K=512, flags=0):
        return lib.fp8_gemm(xq, xs, p, pb, Y, M, N, K, flags, FAKE, 1 << 40, None)
    assert gemm(M=-1) == INV
    assert gemm(M=0) == OK
    assert gemm(xs=None) == INV
    assert gemm(xq=FAKE_MIS) == INV
    assert gemm(Y=FAKE_MIS) == INV
    assert gemm(p=None, M=0) == INV
    assert gemm(flags=0x2) == INV
    assert gemm(flags=0x40) == INV
    assert gemm(K=520) == UNS
    assert gemm(N=0) == INV
    assert gemm(pb=1000) == INV

    def grouped(xq=FAKE, xs=FAKE, p=FAKE, pb=1 << 40, off=FAKE, rows=FAKE, Y=FAKE, R=8, T=4, E=3,
                N=256, K=512, flags=0):
        return lib.fp8_grouped_gemm(xq, xs, p, pb, off, rows, Y, R, T, E, N, K, flags, None)
    assert grouped(off=None) == INV
    assert grouped(off=FAKE_MIS) == INV
    assert grouped(rows=FAKE_MIS) == INV
    assert grouped(rows=None) == INV          # more rows than X has, and no index
    assert grouped(T=0) == INV
    assert grouped(R=0) == OK
    assert grouped(R=0, T=0) == OK
    assert grouped(R=-1) == INV
    assert grouped(E=0) == INV
    assert grouped(K=24) == UNS
    assert grouped(pb=3 * 256 * 512) == INV
    assert grouped(flags=0x4) == INV

    assert lib.fp8_repack(FAKE, None, 1, 256, 128, FAKE, 1 << 30, None) == INV
    assert lib.fp8_repack(FAKE, FAKE, 1, 256, 128, FAKE, 256 * 128, None) == INV
    assert lib.fp8_repack(FAKE, FAKE, 1, 264, 128, FAKE, 1 << 30, None) == UNS
    assert lib.fp8_workspace_bytes(0, 128, 256, 0) == 0
    assert lib.fp8_workspace_bytes(4, 128, 256, 0x40) == 0


def test_rowquant_rejects_before_any_launch(lib):
    def norm(x=FAKE, ldx=256, r=None, ldr=256, w=FAKE, eps=1e-6, h=None, q=FAKE, s=FAKE, T=4,
             W=256, flags=0):
        return lib.rowquant_rmsnorm(x, ldx, r, ldr, w, eps, h, q, s, T, W, flags, None)
    assert norm(T=-1) == INV
    assert norm(T=0) == OK
    assert norm(x=None) == INV
    assert norm(w=None) == INV
    assert norm(s=None) == INV
    assert norm(flags=0x30) == INV            # 16-bit output has no scales
    assert norm(ldx=248) == INV
    assert norm(ldx=260) == INV
    assert norm(r=FAKE, ldr=100) == INV
    assert norm(r=FAKE_MIS) == INV
    assert norm(h=FAKE_MIS) == INV
    assert norm(eps=-1.0) == INV
    assert norm(eps=float("nan")) == INV
    assert norm(W=264, ldx=264) == UNS
    assert norm(W=272, ldx=272, flags=0x20) == UNS
    assert norm(W=131088, ldx=131088) == UNS
    assert norm(flags=0x2) == INV
    assert norm(flags=0x40) == INV

    def swiglu(g=FAKE, ldg=512, u=FAKE, ldu=512, q=FAKE, s=FAKE, T=4, W=256, flags=0):
        return lib.rowquant_swiglu(g, ldg, u, ldu, q, s, T, W, flags, None)
    assert swiglu(T=0) == OK
    assert swiglu(u=None) == INV
    assert swiglu(ldu=128) == INV
    assert swiglu(q=FAKE_MIS) == INV
    assert swiglu(W=100) == UNS
    assert swiglu(W=131088, ldg=131088, ldu=131088, flags=0x10) == UNS


def test_binding_rejects_host_tensors(lib):
    from w4a16_dequant_gemm_amd import fp8, rowquant
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(w4.W4A16Error):
        rowquant.rmsnorm_quantize_rows(x, x[0])
    with pytest.raises(w4.W4A16Error):
        rowquant.swiglu_quantize_rows(x, x)
    with pytest.raises(w4.W4A16Error):
        fp8.fp8_repack(torch.zeros(128, 256, dtype=torch.uint8), torch.zeros(1, 2))
    packed = fp8.PackedFP8(torch.zeros(1, dtype=torch.uint8), 1, 256, 128, False)
    with pytest.raises(w4.W4A16Error):
        fp8.fp8_gemm(torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2), packed)


def test_plan_hint_names(lib):
    from w4a16_dequant_gemm_amd import fp8
    assert fp8.plan_flags_fp8(("tiled", 2)) == 0x20 | (2 << 8)
    with pytest.raises(ValueError):
        fp8.plan_flags_fp8("decode")


def test_limits(lib):
    """The largest row counts and X the kernels' 32-bit counting takes are refused beyond."""
    big = (1 << 30) + 1
    assert lib.fp8_gemm(FAKE, FAKE, FAKE, 1 << 40, FAKE, big, 16, 16, 0, FAKE, 1 << 40, None) == INV
    assert lib.fp8_gemm(FAKE, FAKE, FAKE, 1 << 40, FAKE, 1 << 20, 16, 1 << 17, 0, FAKE, 1 << 40,
                        None) == INV                        # X of 2^37 bytes
    assert lib.fp8_grouped_gemm(FAKE, FAKE, FAKE, 1 << 40, FAKE, FAKE, FAKE, 8, big, 3, 256, 512, 0,
                                None) == INV
    assert lib.fp8_grouped_gemm(FAKE, FAKE, FAKE, 1 << 40, FAKE, FAKE, FAKE, big, 8, 3, 256, 512, 0,
                                None) == INV


@pytest.mark.parametrize("K", [16, 128, 384, 512, 4096, 8208])
def test_workspace_follows_the_plan(lib, K):
    """A hint for the 256 x 256 tile never splits K (nor is taken below four blocks), and a
    split's workspace holds its counters and whole partial tiles."""
    from w4a16_dequant_gemm_amd import fp8
    one = fp8.fp8_workspace_bytes(100, 512, K, fp8.plan_flags_fp8(("tiled", 1)))
    assert one == 0 or K < 512
    assert fp8.fp8_workspace_bytes(100, 512, K, fp8.plan_flags_fp8("stream")) == 0
    small = fp8.fp8_workspace_bytes(100, 512, K, fp8.plan_flags_fp8(("tiled", 3)))
    assert small == 0 or (small - 65536) % (2 * 8 * 64 * 64 * 4) == 0


def test_scales_need_the_alignment_of_a_float(lib):
    """What follows the checks of the pointers is the check of the workspace, so nothing is
    launched."""
    at = lambda n: ctypes.c_void_p(0x10000 + n)                        # noqa: E731
    call = lambda xs: lib.fp8_gemm(FAKE, xs, FAKE, 1 << 40, FAKE, 100, 512, 4096, 0,  # noqa: E731
                                   None, 0, None)
    assert lib.fp8_workspace_bytes(100, 512, 4096, 0) > 0
    for n in (0, 4, 8, 12, 100):
        assert call(at(n)) == w4.W4A16_ERR_WORKSPACE
    for n in (1, 2, 3, 6):
        assert call(at(n)) == INV
        assert lib.fp8_repack(FAKE, at(n), 1, 256, 128, FAKE, 1 << 30, None) == INV
        assert lib.rowquant_swiglu(FAKE, 256, FAKE, 256, FAKE, at(n), 4, 256, 0, None) == INV
        assert lib.rowquant_swiglu(FAKE, 256, FAKE, 256, FAKE, at(n), 4, 256, 0x10, None) == INV


def test_a_split_pays_for_its_partial_tiles(lib):
    """Large products whose partial tiles would make 100 to 210 MB are not split (they are
    faster whole), and no shape of the range asks for more than the parts that still pay."""
    from w4a16_dequant_gemm_amd import fp8
    for M, N, K in ((1425, 11303, 18384), (2113, 7930, 22064), (4073, 1674, 28240),
                    (2028, 8262, 16096)):
        assert fp8.fp8_workspace_bytes(M, N, K) == 0
    import random
    rng = random.Random(3)
    size = lambda low, high: int(low * (high / low) ** rng.random())    # noqa: E731
    split = 0
    for _ in range(4000):
        M, N, K = size(1, 4096), size(64, 28672), size(16, 1792) * 16
        need = fp8.fp8_workspace_bytes(M, N, K)
        # parts beyond 16 MB cost 0.8 us a MB: 96 MB cost 64, more than a split can save
        assert need <= 96 << 20, (M, N, K)
        split += need > 0
    assert split > 1000


@pytest.mark.parametrize("K,parts", [(4096, 8), (8208, 11)])
def test_few_tiles_of_a_long_sum_are_split(lib, K, parts):
    """16 tiles of 64 x 64 leave most of the chip idle unless K is split."""
    from w4a16_dequant_gemm_amd import fp8
    need = fp8.fp8_workspace_bytes(100, 512, K, fp8.plan_flags_fp8(("tiled", 3)))
    assert need == 65536 + 2 * 8 * parts * 64 * 64 * 4
    assert fp8.fp8_workspace_bytes(100, 512, K) > 0
