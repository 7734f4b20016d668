"""The model example (tests/example_model.py) runs; its loss and every gradient agree with the same steps in 64-bit torch."""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, layer

pytestmark = pytest.mark.gpu


def norm(s, w):
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * w


def gated(y, w):
    gate, up = (y @ w.t()).chunk(2, -1)
    return gate * torch.sigmoid(gate) * up


def off(got, want):
    return float(((got.detach().double() - want.detach()).norm() / want.detach().norm()))


def test_example_model():
    _build.build()
    _build.build_layer()
    _build.build_torch()
    import example_model as ex
    p, mixing, collapse, streams, target, loss, rows, scores = ex.main()
    q = {"blocks": [{k: v.detach().double().requires_grad_() for k, v in b.items()} for b in p["blocks"]],
         "norm": p["norm"].detach().double().requires_grad_(), "vocabulary": p["vocabulary"].detach().double().requires_grad_()}
    first = streams.detach().double().requires_grad_()
    s = first
    for b, (pre, post, res) in zip(q["blocks"], mixing):
        x = torch.einsum("tnh,tn->th", s, pre.double())
        z = gated(norm(x, b["norm"]), b["gate_up"]) @ b["down"].t() + x
        s = torch.einsum("tkj,tjh->tkh", res.double(), s) + post.double()[..., None] * z[:, None]
    y = norm(torch.einsum("tnh,tn->th", s, collapse.double()), q["norm"])
    logits = y @ q["vocabulary"].t()
    lse = torch.logsumexp(logits, -1)
    counts = target >= 0
    at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    want = ((lse - at)[counts].sum() + 1e-4 * lse[counts].square().sum()) / counts.sum()
    want.backward()
    # the BF16 steps on the way (about twelve forward, as many backward) round to 2^-9 of a value each
    assert abs(loss.item() - want.item()) <= 2.0 ** -6 * want.item()
    for name, got, ref in [("streams", streams, first), ("norm", p["norm"], q["norm"]), ("vocabulary", p["vocabulary"], q["vocabulary"])] + \
            [(f"{k} {i}", b[k], c[k]) for i, (b, c) in enumerate(zip(p["blocks"], q["blocks"])) for k in b]:
        assert got.grad.shape == got.shape and off(got.grad, ref.grad) < 2.0 ** -5, (name, off(got.grad, ref.grad))
    # 8-bit operands: E4M3 rounds to 2^-4, so the projections are off by a few percent in norm, the logits by less of their spread
    b = q["blocks"][0]
    z = gated(norm(rows.double(), b["norm"]), b["gate_up"]) @ b["down"].t() + rows.double()
    logits = norm(z, q["norm"]) @ q["vocabulary"].t()
    want = torch.logsumexp(logits, -1) - logits.gather(1, target[1:8].clamp(min=0)[:, None])[:, 0]
    assert off(scores, want) < 0.06
    assert layer.wait_timeouts() == 0
