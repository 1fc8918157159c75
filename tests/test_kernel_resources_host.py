"""Registers of kernels that live on having many waves at once, as the compiler reports them
(no GPU): a change that costs waves shows in no result."""
import os
import re
import subprocess

import pytest

from w4a16_dequant_gemm_amd import build as hipbuild


def occupancy(source, defines=()):
    """mangled kernel name -> waves per SIMD"""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("needs hipcc")
    out = subprocess.run([hipcc, *hipbuild.COMMON, *defines, "--cuda-device-only", "-c",
                          "-Rpass-analysis=kernel-resource-usage",
                          os.path.join(hipbuild.CSRC, source), "-o", os.devnull],
                         capture_output=True, text=True, check=True).stderr
    names = re.findall(r"Function Name: (\S+)", out)
    waves = re.findall(r"Occupancy \[waves/SIMD\]: (\d+)", out)
    assert len(names) == len(waves)
    return dict(zip(names, map(int, waves)))


def test_sum_of_rows_keeps_all_its_waves():
    """8 waves a SIMD, the most there are, in both types and for every number of slots: it is
    bound by HBM (fp16 with 8 slots once had 1)."""
    waves = {k: v for k, v in occupancy("combine.hip").items() if "14combine_kernel" in k}
    assert len(waves) == 20       # 2 types, 5 numbers of slots, rows below 8 columns or not
    assert set(waves.values()) == {8}, {k: v for k, v in waves.items() if v < 8}
