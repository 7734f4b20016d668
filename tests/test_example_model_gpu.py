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


def test_two_streams():
    """A gated product and a cross entropy with their gradients on two streams at once: the bytes of each alone."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.25).to(torch.bfloat16)

    x, w, v = normal(700, 1024), normal(2 * 1400, 1024), normal(9001, 1024)
    target = torch.randint(0, 9001, (700,), generator=gen, device="cuda")

    def first():
        y, z = layer.gated_linear_preact(x, w)
        return (y, z, layer.gated_linear(x[:9], w), *layer.gated_linear_backward(y, x, w, z))

    def second():
        loss, lse = layer.linear_cross_entropy(x, v, target)
        return (loss, lse, *layer.linear_cross_entropy(x[:9], v, target[:9]),
                *layer.linear_cross_entropy_backward(loss, x, v, target, lse))

    want = [[t.clone() for t in f()] for f in (first, second)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [[], []]
        for _ in range(10):
            for k, f in enumerate((first, second)):
                with torch.cuda.stream(streams[k]):
                    got[k] = f()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert layer.wait_timeouts() == 0
