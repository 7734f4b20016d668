"""The layer example (tests/example_layer.py) runs, and its steps agree with the same steps in 64-bit torch."""

import math

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, layer

pytestmark = pytest.mark.gpu


def norm(s, w):
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * w


def turn(x, pos, f):
    R = 2 * f.numel()
    angle = pos.double()[:, None, None] * f.double()
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)


def close(got, want, what, most):
    off = (got.double() - want).norm() / want.norm()
    assert off < most, (what, float(off))


def test_example_layer():
    _build.build()
    _build.build_layer()
    _build.build_torch()
    import example_layer as ex
    p, streams, pre, out, qk, z, qkv, row, carried = ex.main()
    assert tuple(out.shape) == (ex.T, ex.n, ex.H) and tuple(qk.shape) == (ex.T, 2 * ex.heads, ex.D)
    # every BF16 step rounds to 2^-9 of a value: a chain of five stays within 2^-6 in norm
    q = {k: v.detach().double() for k, v in p.items()}
    x = torch.einsum("tnh,tn->th", streams.detach().double(), pre.detach().double())
    y = norm(x, q["norm"])
    f = layer.rotary_frequencies(ex.D, scaling="yarn", factor=4.0)
    want = turn((y @ q["qkv"].t())[:, :2 * ex.heads * ex.D].unflatten(1, (2 * ex.heads, ex.D)),
                torch.arange(ex.T, device="cuda"), f)
    close(qk, want, "queries and keys", 2.0 ** -6)
    for name, t in {**p, "streams": streams, "pre": pre}.items():
        assert t.grad is not None and t.grad.shape == t.shape and torch.isfinite(t.grad.float()).all(), name
        assert t.grad.float().abs().max() > 0, name
    # the 8-bit decode: E4M3 rounds to 2^-4, so each product is off by a few percent in norm
    s = row.double() + carried.double()
    y = norm(s, q["norm"])
    want = y @ q["qkv"].t()
    half = 2 * ex.heads * ex.D
    close(qkv[:, half:], want[:, half:], "values", 0.06)
    close(qkv[:, :half].unflatten(1, (2 * ex.heads, ex.D)),
          turn(want[:, :half].unflatten(1, (2 * ex.heads, ex.D)), torch.tensor([5, 70, 100000], device="cuda"), f),
          "rotated", 0.06)
    up = y @ q["up"].t()
    up = up * 0.5 * (1 + torch.erf(up * math.sqrt(0.5)))
    close(z, up @ q["down"].t() + s, "layer output", 0.06)
