"""Second derivatives through the layer's autograd functions on a GPU: rotary's
are right, the others' are refused."""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, autograd, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()


def normal(seed, *shape, dtype=torch.float16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_twice(interleaved):
    T, heads, D, scale = 9, 3, 16, 0.5
    x = normal(1, T, heads, D).requires_grad_()
    pos, f = torch.arange(T, device="cuda") * 100, layer.rotary_frequencies(D - 4)

    def plain(v):
        R = D - 4
        angle = pos.double()[:, None] * f.double()
        c, s = (angle.cos() * scale)[:, None], (angle.sin() * scale)[:, None]
        a, b = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
        p, q = a * c - b * s, b * c + a * s
        turned = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
        return torch.cat([turned, v[..., R:]], -1)

    def penalty(call, v):
        loss = call(v).pow(3).sum()
        grad, = torch.autograd.grad(loss, v, create_graph=True)
        return torch.autograd.grad(loss + grad.pow(2).sum(), v)[0]

    got = penalty(lambda v: autograd.rotary(v, pos, f, interleaved=interleaved, scale=scale), x)
    want = penalty(plain, x.detach().double().requires_grad_())
    # about a dozen roundings to 11 bits, in the norm
    assert (got.double() - want).norm() <= 16 * 2.0 ** -11 * want.norm()


def test_the_others_refuse():
    x, w, wn = normal(2, 5, 64).requires_grad_(), normal(3, 8, 64).requires_grad_(), torch.ones(64, device="cuda").requires_grad_()
    for call in (lambda: autograd.linear(x, w), lambda: autograd.rms_norm(x, wn)[0], lambda: autograd.rms_norm(x, wn, residual=x)[1]):
        loss = call().float().sum()
        grad, = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError, match="once"):
            (loss + grad.float().pow(2).sum()).backward()
