"""A warp's bounded wait whose lanes disagree: all of them give up."""

import ctypes
import os
import subprocess

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_warp_gives_up_together(tmp_path):
    so = str(tmp_path / "layer_warp_probe.so")
    cmd = [_build.nvcc_path(), *_build.NVCC_FLAGS, "-shared", "-I", _build.CSRC, "-o", so,
           os.path.join(HERE, "layer_warp_probe.cu")]
    subprocess.run(cmd, check=True, capture_output=True)
    probe = ctypes.CDLL(so)
    probe.run_warp_probe.argtypes = [ctypes.c_void_p]
    probe.run_warp_probe.restype = ctypes.c_int
    result = torch.full((32,), 7, dtype=torch.int32, device="cuda")
    assert probe.run_warp_probe(result.data_ptr()) == 0
    assert result.tolist() == [0] * 32
