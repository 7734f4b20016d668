"""The autograd functions of the gated product and the cross entropy on the
host: batches and weights of unusual shapes, with the kernels' calls replaced
by torch formulas."""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import autograd, layer

B = torch.bfloat16


@pytest.fixture
def formulas(monkeypatch):
    def gated(x, w, bias=None, activation="silu", stream=None):
        z = x.float() @ w.float().t()
        F = w.shape[0] // 2
        return (z[:, :F] * z[:, F:]).to(x.dtype), z.to(x.dtype)

    def gated_backward(g, x, w, z, activation="silu", bias=True, want=(True, True), stream=None):
        F = w.shape[0] // 2
        u = torch.cat([g * z[:, F:], g * z[:, :F]], 1)
        return u @ w if want[0] else None, u.t() @ x if want[1] else None, u.float().sum(0) if bias else None

    def entropy(x, w, target, stream=None):
        z = x.float() @ w.float().t()
        lse = torch.logsumexp(z, -1)
        return lse - z.gather(1, target[:, None])[:, 0], lse

    def entropy_backward(gl, x, w, target, lse, grad_lse=None, want=(True, True), stream=None):
        return torch.ones_like(x) if want[0] else None, torch.ones_like(w) if want[1] else None

    monkeypatch.setattr(layer, "gated_linear_preact", gated)
    monkeypatch.setattr(layer, "gated_linear", lambda *a, **k: gated(*a, **k)[0])
    monkeypatch.setattr(layer, "gated_linear_backward", gated_backward)
    monkeypatch.setattr(layer, "linear_cross_entropy", entropy)
    monkeypatch.setattr(layer, "linear_cross_entropy_backward", entropy_backward)


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 3)])
def test_no_tokens(formulas, lead):
    x, w = torch.empty(*lead, 8, dtype=B), torch.ones(10, 8, dtype=B)
    assert autograd.gated_linear(x, w).shape == (*lead, 5)                  # no gradient: z is not kept
    with torch.no_grad():
        assert autograd.gated_linear(x, w.requires_grad_()).shape == (*lead, 5)
    x.requires_grad_()
    y = autograd.gated_linear(x, w)
    assert y.shape == (*lead, 5)
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape and (w.grad == 0).all()
    loss, lse = autograd.linear_cross_entropy(x, w, torch.empty(lead, dtype=torch.int64))
    assert loss.shape == lse.shape == lead
    (loss.sum() + lse.sum()).backward()
    assert x.grad.shape == x.shape


@pytest.mark.parametrize("shape", [(8,), (2, 5, 8), (1, 10, 8)])
def test_a_weight_has_two_dimensions(formulas, shape):
    """Refused where it is given, not by the gradient's shape in the backward."""
    x, w = torch.ones(3, 8, dtype=B).requires_grad_(), torch.ones(*shape, dtype=B).requires_grad_()
    with pytest.raises(ValueError, match="weight must be 2-d"):
        autograd.gated_linear(x, w)
    with pytest.raises(ValueError, match="weight must be 2-d"):
        autograd.linear_cross_entropy(x, w, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="weight must be 2-d"), torch.no_grad():
        autograd.gated_linear(x, w)
