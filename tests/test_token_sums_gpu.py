"""Weight gradients of very many tokens, all terms of one sign: the tensor cores cut off each addition's last bits, so that
a sum falls short by a part that grows with the terms that one accumulator takes.  That is at most 16384 (sums of runs meet in
FP32, rounded to nearest), whatever the number of tokens: the bound does not grow with it but for those additions.

The gradients of the logits (and u) are powers of two here, and x has 11 bits, so every product is exact.
"""

import math

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, layer

pytestmark = pytest.mark.gpu

RUN = 16384
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()
    yield
    assert layer.wait_timeouts() == 0


def bound(T, want, dtype):
    """16 products at a time, truncated (as test_entropy_gpu.py counts them), in runs; the runs' additions; the rounding."""
    return (1.2 * (2 * math.ceil(min(T, RUN) / 16) + 32) * 2.0 ** -23 + math.ceil(T / RUN) * 2.0 ** -24 + U[dtype]) * want


def ones_to_two(T, I, dtype, seed):
    """Values of 1 .. 2 in all of the type's bits, made a part at a time."""
    x = torch.empty(T, I, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for part in x.split(1 << 18):
        part.copy_(1 + torch.rand(part.shape, generator=g, device="cuda"))
    return x.clamp_(max=2 - 2 * U[dtype])


def columns(x, factor):
    return sum((part.double() * f[:, None]).sum(0) for part, f in zip(x.split(1 << 18), factor.double().split(1 << 18)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("I", [16, 17])          # by rows, and with its values on the lanes
@pytest.mark.parametrize("T", [65536, (1 << 21) + 77])
def test_cross_entropy(T, I, dtype):
    V = 8
    x = ones_to_two(T, I, dtype, I)
    w = torch.zeros(V, I, dtype=dtype, device="cuda")
    target = torch.full((T,), -100, device="cuda")
    _, lse = layer.linear_cross_entropy(x, w, target)
    gs = torch.full((T,), 8.0 / 2 ** 21, device="cuda")
    _, gw = layer.linear_cross_entropy_backward(None, x, w, target, lse, grad_lse=gs, want=(False, True))
    want = columns(x, gs / V)[None].expand(V, -1)       # every probability is 1/8, up to what its rounding takes away
    off = (gw.double() - want).abs()
    assert (off <= bound(T, want, dtype)).all(), float((off / want).max())


# parts of K in a cluster's CTAs; tiles for every pair, off 16 bytes and by rows
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,I,F", [(65536, 16, 24), (65536, 264, 160), ((1 << 22) + 77, 16, 24), (1 << 20, 264, 160), (1 << 20, 17, 3),
                                   ((1 << 20) + 5, 600, 300), (1 << 20, 1279, 2100), (1 << 20, 1040, 2100)])
def test_gated(T, I, F, dtype):
    x = ones_to_two(T, I, dtype, I)
    w = torch.zeros(2 * F, I, dtype=dtype, device="cuda")
    z, gy = torch.ones(T, 2 * F, dtype=dtype, device="cuda"), torch.full((T, F), 2.0 ** -12, dtype=dtype, device="cuda")
    _, gw, _ = layer.gated_linear_backward(gy, x, w, z, activation="relu", bias=False, want=(False, True))
    want = columns(x, torch.full((T,), 2.0 ** -12, device="cuda"))[None].expand(2 * F, -1)
    off = (gw.double() - want).abs()
    assert (off <= bound(T, want, dtype)).all(), float((off / want).max())
