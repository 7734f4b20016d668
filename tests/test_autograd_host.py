"""The autograd functions' own part, without a GPU: the kernels' calls are
replaced by torch formulas in the inputs' type."""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import autograd, binding, layer

B = torch.bfloat16


def norm(x, w, residual=None, eps=1e-6, stream=None):
    total = x if residual is None else x + residual
    rstd = torch.rsqrt(total.float().square().mean(-1) + eps)
    return (total.float() * rstd[:, None] * w).to(x.dtype), total, rstd


def norm_backward(g, s, w, rstd, grad_total=None, stream=None):
    n, u = s.float() * rstd[:, None], g.float() * w
    gx = rstd[:, None] * (u - n * (u * n).mean(-1, keepdim=True))
    return (gx if grad_total is None else gx + grad_total.float()).to(s.dtype), (g.float() * n).sum(0)


def product(x, w, bias=None, activation="none", residual=None, stream=None):
    z = x.float() @ w.float().t() + (0 if bias is None else bias)
    y = torch.relu(z) if activation == "relu" else z
    return (y if residual is None else y + residual.float()).to(x.dtype)


def product_preact(x, w, bias=None, activation="none", residual=None, stream=None):
    return product(x, w, bias, activation, residual), product(x, w, bias)


def product_backward(g, x, w, z=None, activation="none", bias=True, want=(True, True), stream=None):
    u = g.float() * (z > 0) if activation == "relu" else g.float()
    return ((u @ w.float()).to(x.dtype) if want[0] else None, (u.t() @ x.float()).to(x.dtype) if want[1] else None,
            u.sum(0) if bias else None)


@pytest.fixture(autouse=True)
def formulas(monkeypatch):
    monkeypatch.setattr(layer, "rms_norm", norm)
    monkeypatch.setattr(layer, "rms_norm_backward", norm_backward)
    monkeypatch.setattr(layer, "linear", product)
    monkeypatch.setattr(layer, "linear_preact", product_preact)
    monkeypatch.setattr(layer, "linear_backward", product_backward)
    monkeypatch.setattr(layer, "rotary", lambda x, p, f, interleaved=False, scale=1.0, inverse=False: x * scale)
    monkeypatch.setattr(binding, "aggregate", lambda r, p: (r.float() * p[..., None]).sum(1).to(r.dtype))
    monkeypatch.setattr(binding, "aggregate_sigmoid", lambda r, m, a, b: r.sum(1))
    monkeypatch.setattr(binding, "post", lambda x, y, p, r: x * 2)
    monkeypatch.setattr(binding, "post_sigmoid", lambda x, y, m, a, b, r: x * 2)
    monkeypatch.setattr(binding, "aggregate_backward", lambda g, r, p: (
        (g[:, None].float() * p[..., None]).to(r.dtype), (g[:, None].float() * r.float()).sum(-1)))
    monkeypatch.setattr(binding, "aggregate_sigmoid_backward", lambda g, r, m, a, b: (
        torch.zeros_like(r), torch.zeros_like(m), torch.zeros_like(m)))
    monkeypatch.setattr(binding, "post_backward", lambda g, x, y, p, r: tuple(torch.zeros_like(t) for t in (x, y, p, r)))
    monkeypatch.setattr(binding, "post_sigmoid_backward", lambda g, x, y, m, a, b, r: tuple(
        torch.zeros_like(t) for t in (x, y, m, m, r)))
    monkeypatch.setattr(binding, "sigmoid_param_grad", lambda z, m: (torch.zeros(m.shape[-1]), torch.zeros(1)))


def bf(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(B).requires_grad_()


def fp(*shape):
    return torch.rand(*shape, generator=torch.Generator().manual_seed(sum(shape))).requires_grad_()


CALLS = {
    "rms_norm": lambda: (lambda x, w: autograd.rms_norm(x, w)[0], bf(5, 8), fp(8)),
    "rms_norm_residual": lambda: (lambda x, w, r: autograd.rms_norm(x, w, residual=r)[1], bf(5, 8), fp(8), bf(5, 8)),
    "linear": lambda: (autograd.linear, bf(5, 8), bf(6, 8)),
    "linear_relu": lambda: (lambda x, w, b: autograd.linear(x, w, b, "relu"), bf(5, 8), bf(6, 8), fp(6)),
    "rotary": lambda: (lambda x: autograd.rotary(x, torch.arange(5), torch.ones(4), scale=2.0), bf(5, 2, 8)),
    "h_aggregate": lambda: (autograd.h_aggregate, bf(5, 4, 8), fp(5, 4)),
    "h_aggregate_sigmoid": lambda: (autograd.h_aggregate_sigmoid, bf(5, 4, 8), fp(5, 4), fp(1), fp(4)),
    "mhc_post": lambda: (autograd.mhc_post, bf(5, 4, 8), bf(5, 8), fp(5, 4), fp(5, 4, 4)),
    "mhc_post_sigmoid": lambda: (autograd.mhc_post_sigmoid, bf(5, 4, 8), bf(5, 8), fp(5, 4), fp(1), fp(4), fp(5, 4, 4)),
}


@pytest.mark.parametrize("power", [1, 3])
@pytest.mark.parametrize("name", [n for n in CALLS if n != "rotary"])
def test_second_derivatives_are_refused(name, power):
    """A gradient penalty raises; without its term the weights' gradients would silently lack it.  (power 1: the
    gradient that reaches the function is a constant and requires none itself.)"""
    f, *args = CALLS[name]()
    loss = f(*args).float().pow(power).sum()
    grad, = torch.autograd.grad(loss, args[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        (loss + grad.float().square().sum()).backward()


@pytest.mark.parametrize("name", CALLS)
def test_create_graph_keeps_first_derivatives(name):
    f, *args = CALLS[name]()
    want = torch.autograd.grad(f(*args).float().square().sum(), args)
    got = torch.autograd.grad(f(*args).float().square().sum(), args, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t in args:
        t.grad = None
    f(*args).float().square().sum().backward()
    assert all(torch.equal(t.grad, b) and not t.grad.requires_grad for t, b in zip(args, want))


def test_rotary_second_derivative():
    """The rotation is linear: its gradient is a rotation too and has one of its own (the stand-in for the kernel
    multiplies by 2 both ways, so loss = sum (2x)^3, grad = 24 x^2, penalty = sum grad^2)."""
    f, x = CALLS["rotary"]()
    x = x.detach().mul(4).round().div(4).requires_grad_()          # products exact in 8 bits or nearly so
    loss = f(x).float().pow(3).sum()
    grad, = torch.autograd.grad(loss, x, create_graph=True)
    got, = torch.autograd.grad(grad.float().square().sum(), x)
    want = 4 * 24 ** 2 * x.detach().double() ** 3
    # four roundings to 8 bits on the way
    assert ((got.double() - want).abs() <= 4 * 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_outputs_without_a_gradient(with_residual, monkeypatch):
    """An unused output's gradient is not made up of zeros: the kernel then reads one input less."""
    seen = []
    monkeypatch.setattr(layer, "rms_norm_backward", lambda g, s, w, rstd, grad_total=None, stream=None: (
        seen.append(grad_total), norm_backward(g, s, w, rstd, grad_total))[1])
    x, w, r = bf(3, 5, 8), fp(8), bf(3, 5, 8) if with_residual else None
    args = [x, w] + [r] * with_residual

    def grads(loss):
        return torch.autograd.grad(loss, args)

    y, total = autograd.rms_norm(x, w, residual=r)
    only_y = grads(y.float().square().sum())
    assert seen == [None] and only_y[0].shape == x.shape
    y, total = autograd.rms_norm(x, w, residual=r)
    both = grads(y.float().square().sum() + total.float().square().sum())
    assert len(seen) == 2 and torch.equal(seen[1], 2 * total.detach().reshape(-1, 8))
    assert not torch.equal(both[0], only_y[0]) and torch.equal(both[1], only_y[1])
    y, total = autograd.rms_norm(x, w, residual=r)
    only_total = torch.autograd.grad(total.float().square().sum(), args, allow_unused=True)
    assert torch.equal(only_total[0], 2 * total.detach()) and (only_total[1] is None or not only_total[1].any())
    given = torch.ones_like(total)
    torch.autograd.backward([autograd.rms_norm(x, w, residual=r)[1]], [given])
    x.grad.zero_()                                     # the caller's tensor is not handed on
    assert (given == 1).all()
    if with_residual:
        assert torch.equal(only_total[2], only_total[0]) and torch.equal(only_y[2], only_y[0])


@pytest.fixture
def strict(formulas, monkeypatch):
    """The stand-ins refuse what the kernels' calls refuse: rows that are not contiguous or share memory."""
    def rows(t):
        assert t is None or t.dim() != 2 or ((t.stride(1) == 1 or t.shape[1] == 1) and (t.stride(0) >= t.shape[1] or t.shape[0] == 1))

    def product_strict(f):
        def call(x, w, bias=None, activation="none", residual=None, stream=None):
            for t in (x, w, residual):
                rows(t)
            assert bias is None or bias.is_contiguous()
            return f(x, w, bias, activation, residual)
        return call

    def norm_strict(x, w, residual=None, eps=1e-6, stream=None):
        rows(x), rows(residual)
        assert w.is_contiguous()
        return norm(x, w, residual, eps)

    def rotary_strict(x, p, f, interleaved=False, scale=1.0, inverse=False):
        assert x.stride(2) == 1 and 0 not in x.stride()
        return x * scale

    monkeypatch.setattr(layer, "rms_norm", norm_strict)
    monkeypatch.setattr(layer, "linear", product_strict(product))
    monkeypatch.setattr(layer, "linear_preact", product_strict(product_preact))
    monkeypatch.setattr(layer, "rotary", rotary_strict)


def layouts(*shape):
    """The same shape transposed in memory, and broadcast over the rows."""
    return {"transposed": bf(*shape[:-2], shape[-1], shape[-2]).detach().transpose(-1, -2),
            "broadcast": bf(shape[-1]).detach().expand(*shape)}


@pytest.mark.parametrize("layout", ["transposed", "broadcast"])
def test_layouts_of_inputs(layout, strict):
    x, r, big = layouts(6, 8)[layout], layouts(6, 8)[layout], layouts(3, 6, 8)[layout]
    w = torch.rand(16)[::2]
    for a, b in ((autograd.rms_norm(x, w, residual=r), autograd.rms_norm(x.contiguous(), w.contiguous(), residual=r.contiguous())),
                 (autograd.rms_norm(big, w, residual=big), autograd.rms_norm(big.contiguous(), w, residual=big.contiguous()))):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    wl, bias, out = bf(5, 8).detach(), torch.rand(10)[::2], layouts(6, 5)[layout]
    for act in ("none", "relu"):
        got = autograd.linear(x, wl, bias=bias, activation=act, residual=out)
        assert torch.equal(got, autograd.linear(x.contiguous(), wl, bias=bias.contiguous(), activation=act, residual=out.contiguous()))
    q = layouts(4, 2, 8)[layout]
    assert torch.equal(autograd.rotary(q, torch.arange(4), torch.ones(4), scale=2.0), q * 2)
    # gradients come in the inputs' shapes
    x.requires_grad_(), r.requires_grad_()
    y, total = autograd.rms_norm(x, w, residual=r)
    (autograd.linear(y, wl, residual=out).float().sum() + total.float().sum()).backward()
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
