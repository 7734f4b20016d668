"""The bounded waits of the layer operators' kernels: a wait that nothing ends
gives up after about 1 s and reports it; normal runs record none."""

import ctypes
import os
import subprocess

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, layer

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("layer_wait_probe") / "layer_wait_probe.so")
    cmd = [_build.nvcc_path(), *_build.NVCC_FLAGS, "-shared", "-I", _build.CSRC, "-o", so,
           os.path.join(HERE, "layer_wait_probe.cu")]
    subprocess.run(cmd, check=True, capture_output=True)
    p = ctypes.CDLL(so)
    p.run_wait_probe.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    p.run_wait_probe.restype = ctypes.c_int
    return p


@pytest.mark.parametrize("arrive", [1, 0])
def test_bounded_wait(probe, arrive):
    result = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    elapsed = torch.zeros((1,), dtype=torch.int64, device="cuda")
    assert probe.run_wait_probe(arrive, result.data_ptr(), elapsed.data_ptr()) == 0
    assert int(result.item()) == arrive
    if arrive:
        assert int(elapsed.item()) < 10_000_000
    else:
        assert 1_000_000_000 <= int(elapsed.item()) < 5_000_000_000


def test_no_timeouts_in_normal_runs():
    _build.build_layer()
    assert layer.wait_timeouts() >= 0    # reset
    x, w = torch.ones(700, 1280, device="cuda").bfloat16(), torch.ones(1280, device="cuda")
    wl = torch.ones(2048, 1280, device="cuda").bfloat16()
    for rows in (1, 700):
        y, total, rstd = layer.rms_norm(x[:rows], w)
        layer.rms_norm_backward(y, total, w, rstd)
        z = layer.linear(y, wl)
        layer.linear_backward(z, y, wl)
    assert layer.wait_timeouts() == 0
