"""The gated product on a GPU against its definition in 64 bits.

Tolerances: a product's FP32 sums are off by SUMS of the magnitudes of their
terms (truncating additions in the tensor cores, 16 products at a time, and the
products' own alignment), an FP32 step by 2^-24, a result rounded to p bits by
2^-p of itself (twice the half step, for results next to a rounding boundary).
The activations have slopes of at most 1.13 and FP32 errors of 2^-18 of
max(1, |z|).
"""

import math

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, autograd, layer

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
BOTH = [BF, HF]
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}
TINY = {BF: 2.0 ** -133, HF: 2.0 ** -24}
E = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu"]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()
    yield
    assert layer.wait_timeouts() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, spread=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * spread).to(dtype)


def within(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    n = int(bad.sum())
    assert n == 0, f"{what}: {n} of {bad.numel()} outside, worst {float((off - bound).max()):.3g} over"


def strided(t, extra=8, lead=0):
    rows, length = t.shape
    b = torch.full((rows, lead + length + extra), float("nan"), device="cuda").to(t.dtype)
    b[:, lead:lead + length] = t
    return b[:, lead:lead + length]


def sums(K, size):
    return 1.2 * (2 * math.ceil(K / 16) + 32) * 2.0 ** -23 * size


def act_ref(z, kind):
    """(act(z), act'(z))"""
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if kind == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def case(T, I, F, dtype, bias, seed=0, fp8=False):
    g = gen(T + 7 * I + 13 * F + seed)
    x, w = normal(g, T, I), normal(g, 2 * F, I, spread=I ** -0.5)
    sx = sw = None
    if fp8:
        sx, sw = x.abs().amax(-1) / 448, w.abs().amax(-1) / 448
        x, w = ((a / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for a, s in ((x, sx), (w, sw)))
    else:
        x, w = x.to(dtype), w.to(dtype)
    b = normal(g, 2 * F) if bias else None
    x64, w64 = x.double(), w.double()
    if fp8:
        x64, w64 = x64 * sx.double()[:, None], w64 * sw.double()[:, None]
    z = x64 @ w64.t() + (0 if b is None else b.double())
    off = sums(I, x64.abs() @ w64.abs().t()) + 4 * E * (z.abs() + 1)
    return x, sx, w, sw, b, z, off


def check(y, z, off, act, dtype, what="y"):
    F = z.shape[1] // 2
    gate, up = z[:, :F], z[:, F:]
    dg, du = off[:, :F], off[:, F:]
    a, _ = act_ref(gate, act)
    da = 1.13 * dg + 2.0 ** -18 * (1 + gate.abs())
    want = a * up
    within(y, want, da * up.abs() + a.abs() * du + da * du + (U[dtype] + E) * want.abs() + TINY[dtype], what)


SIZES = [(1, 2048, 8192), (1, 64, 8), (1, 1, 1), (2, 8, 24), (3, 100, 65), (16, 128, 64), (17, 256, 63), (64, 520, 150),
         (129, 1279, 257), (200, 64, 1024), (256, 192, 128), (257, 320, 20), (300, 1024, 260), (513, 72, 500),
         (1000, 640, 133), (2049, 328, 1300), (700, 2048, 1100)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,I,F", SIZES)
def test_forward(T, I, F, dtype):
    for act, bias in (("silu", False), ("gelu", True)):
        x, _, w, _, b, z, off = case(T, I, F, dtype, bias)
        check(layer.gated_linear(x, w, bias=b, activation=act), z, off, act, dtype)
        y, got_z = layer.gated_linear_preact(x, w, bias=b, activation=act)
        check(y, z, off, act, dtype)
        within(got_z, z, off + U[dtype] * z.abs() + TINY[dtype], "z")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [5, 600])
def test_activations(T, act):
    x, _, w, _, b, z, off = case(T, 264, 1150, BF, True)
    check(layer.gated_linear(x, w, bias=b, activation=act), z, off, act, BF)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,I,F", [(1, 7168, 256), (1, 16, 8), (3, 17, 5), (64, 512, 150), (129, 1280, 257), (700, 1000, 130),
                                   (2049, 336, 1300)])
def test_forward_fp8(T, I, F, dtype):
    x, sx, w, sw, b, z, off = case(T, I, F, dtype, True, fp8=True)
    check(layer.gated_linear_fp8(x, sx, w, sw, bias=b, dtype=dtype), z, off, "silu", dtype)
    check(layer.gated_linear_fp8(x, sx[:, None], w, sw[:, None], bias=b, dtype=dtype), z, off, "silu", dtype)


def test_values_are_the_products_own():
    """Bit for bit: z is what `linear` gives, and y follows from the unrounded z."""
    for T, I, F in ((1, 4096, 300), (40, 1024, 700), (600, 2048, 520)):
        x, _, w, _, b, z, off = case(T, I, F, BF, True)
        y, got_z = layer.gated_linear_preact(x, w, bias=b, activation="relu")
        assert torch.equal(got_z, layer.linear_preact(x, w, bias=b, activation="relu")[1])
        assert (y[got_z[:, :F] < 0] == 0).all()


@pytest.mark.parametrize("lead,extra", [(0, 8), (8, 8), (1, 0), (0, 1), (3, 5)])
def test_strides(lead, extra):
    x, _, w, _, b, z, off = case(37, 200, 166, BF, True)
    want = layer.gated_linear_preact(x, w, bias=b)
    got = layer.gated_linear_preact(strided(x, extra, lead), strided(w, extra, lead), bias=b)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    g = gen(3)
    gy = normal(g, 37, 166, dtype=BF)
    want = layer.gated_linear_backward(gy, x, w, want[1])
    got = layer.gated_linear_backward(gy, strided(x, extra, lead), strided(w, extra, lead), got[1])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("I,F", [(7168, 1024), (4096, 3600), (1024, 512), (1279, 150), (512, 12), (520, 8200), (256, 5001)])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_do_not_depend_on_the_batch(I, F, fp8):
    if fp8:
        I = I // 16 * 16
    T = 1500
    x, sx, w, sw, b, *_ = case(T, I, F, BF, True, fp8=fp8)

    def run(lo, hi):
        if fp8:
            return layer.gated_linear_fp8(x[lo:hi], sx[lo:hi], w, sw, bias=b)
        return layer.gated_linear(x[lo:hi], w, bias=b)

    whole = run(0, T)
    assert torch.equal(run(0, T), whole)
    for lo, hi in ((0, 1), (777, 778), (1499, 1500), (3, 40), (100, 229), (640, 940), (0, 700), (5, 21), (5, 22), (5, 37), (5, 38),
                   (5, 69), (5, 70)):
        assert torch.equal(run(lo, hi), whole[lo:hi]), (lo, hi)


def test_rows_with_nan_and_infinities():
    """They stay in their rows, also next to ragged edges; nothing past the outputs is written."""
    x, _, w, _, _, z, off = case(70, 100, 75, BF, False)
    x[3, 7] = float("nan")
    x[69, 99] = float("inf")
    y = layer.gated_linear(x, w)
    keep = [i for i in range(70) if i not in (3, 69)]
    check(y[keep], z[keep], off[keep], "silu", BF)
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[69].float()).all()
    # a weight's row past the gate's is the up projection's, not a stray one
    w2 = w.clone()
    w2[74] = float("nan")
    y = layer.gated_linear(x[:3], w2)
    assert torch.isnan(y[:, 74]).all() and torch.isfinite(y[:, :74].float()).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,I,F", [(1, 64, 8), (1, 1, 1), (3, 100, 65), (65, 256, 64), (129, 1279, 257), (300, 520, 12),
                                   (2049, 328, 1300), (700, 72, 1100)])
def test_backward(T, I, F, act, dtype):
    g = gen(T + I + F)
    x, w = normal(g, T, I, dtype=dtype), normal(g, 2 * F, I, dtype=dtype, spread=F ** -0.5)
    z, gy = normal(g, T, 2 * F, dtype=dtype), normal(g, T, F, dtype=dtype)
    gate, up, g64 = z[:, :F].double(), z[:, F:].double(), gy.double()
    a, s = act_ref(gate, act)
    u = torch.cat([g64 * up * s, g64 * a], 1)
    # the slope and the activation to 2^-18 of max(1, |z|), two products; then u's rounding
    fine = torch.cat([(g64 * up).abs(), g64.abs()], 1) * 2.0 ** -18 * (1 + gate.abs().repeat(1, 2)) + 4 * E * u.abs()
    coarse = fine + 1.01 * U[dtype] * u.abs() + TINY[dtype]
    got = layer.gated_linear_backward(gy, x, w, z, activation=act)
    want, size = u @ w.double(), u.abs() @ w.double().abs()
    within(got[0], want, sums(2 * F, size) + coarse @ w.double().abs() + U[dtype] * want.abs() + TINY[dtype], "grad_x")
    want, size = u.t() @ x.double(), u.abs().t() @ x.double().abs()
    within(got[1], want, sums(T, size) + coarse.t() @ x.double().abs() + U[dtype] * want.abs() + TINY[dtype], "grad_w")
    chain = math.ceil(T / 64) + 72
    within(got[2], u.sum(0), chain * E * u.abs().sum(0) + fine.sum(0) + 1e-30, "grad_b")
    # each gradient alone has the same bits
    one = layer.gated_linear_backward(gy, x, w, z, activation=act, bias=False, want=(True, False))
    assert one[1] is None and one[2] is None and torch.equal(one[0], got[0])
    one = layer.gated_linear_backward(gy, x, w, z, activation=act, bias=False, want=(False, True))
    assert one[0] is None and torch.equal(one[1], got[1])
    one = layer.gated_linear_backward(gy, x, w, z, activation=act, want=(False, False))
    assert torch.equal(one[2], got[2])


def test_grad_x_does_not_depend_on_the_batch():
    g = gen(11)
    T, I, F = 900, 1024, 700
    x, w = normal(g, T, I, dtype=BF), normal(g, 2 * F, I, dtype=BF)
    z, gy = normal(g, T, 2 * F, dtype=BF), normal(g, T, F, dtype=BF)
    whole = layer.gated_linear_backward(gy, x, w, z, bias=False, want=(True, False))[0]
    for lo, hi in ((0, 1), (3, 40), (640, 900)):
        part = layer.gated_linear_backward(gy[lo:hi], x[lo:hi], w, z[lo:hi], bias=False, want=(True, False))[0]
        assert torch.equal(part, whole[lo:hi]), (lo, hi)


@pytest.mark.parametrize("T,D", [(40, 328), (700, 520), (2049, 1032), (300, 1023)])
def test_calls_in_a_row_and_in_a_graph(T, D):
    """The kernels of consecutive calls overlap; memory that one frees is the next one's."""
    g = gen(T + D)
    w = [normal(g, 2 * D, D, dtype=BF, spread=D ** -0.5) for _ in range(4)]
    first = normal(g, T, D, dtype=BF)

    def chain(wait):
        x, out = first, []
        for weight in w:
            y, z = layer.gated_linear_preact(x, weight)
            wait()
            got = layer.gated_linear_backward(y, x, weight, z)
            wait()
            out += [y, z, *got]
            x = y
        return out

    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,I,F", [(7550, 383, 136), (5000, 1024, 24), (40, 520, 9000)])
def test_many_calls_in_a_row(T, I, F):
    """Thousands of calls whose kernels overlap all give the same bytes, and each of them ends."""
    x, _, w, _, b, z, off = case(T, I, F, BF, False)
    want = layer.gated_linear(x, w, activation="relu")
    check(want, z, off, "relu", BF)
    torch.cuda.synchronize()
    for _ in range(40):
        for _ in range(100):
            got = layer.gated_linear(x, w, activation="relu")
        assert torch.equal(got, want)


def test_other_stream():
    x, _, w, _, b, z, off = case(300, 511, 350, BF, True)      # (odd rows: a workspace)
    want = layer.gated_linear_preact(x, w, bias=b)
    gy = normal(gen(1), 300, 350, dtype=BF)
    want_g = layer.gated_linear_backward(gy, x, w, want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer.gated_linear_preact(x, w, bias=b)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    got = layer.gated_linear_preact(x, w, bias=b, stream=side)
    got_g = layer.gated_linear_backward(gy, x, w, got[1], stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got, *got_g), (*want, *want_g)))


def test_no_tokens():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(16, 64, dtype=BF, device="cuda")
    assert layer.gated_linear(x, w).shape == (0, 8)
    y, z = layer.gated_linear_preact(x, w)
    assert z.shape == (0, 16)
    gx, gw, gb = layer.gated_linear_backward(y, x, w, z)
    assert gx.shape == (0, 64) and gw.shape == (16, 64) and (gw == 0).all() and (gb == 0).all()


def test_refusals():
    x, w = torch.ones(4, 64, dtype=BF, device="cuda"), torch.ones(16, 64, dtype=BF, device="cuda")
    y, z = layer.gated_linear_preact(x, w)
    s = torch.ones(4, device="cuda")
    for bad in (lambda: layer.gated_linear(x.float(), w), lambda: layer.gated_linear(x, w.half()), lambda: layer.gated_linear(None, w),
                lambda: layer.gated_linear(x, w, bias=torch.ones(16, device="cuda", dtype=BF)),
                lambda: layer.gated_linear_fp8(x, s, w, s), lambda: layer.gated_linear_fp8(x, None, w, s),
                lambda: layer.gated_linear_backward(y, x, w, None), lambda: layer.gated_linear_backward(y.half(), x, w, z)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: layer.gated_linear(x, w[:15]), lambda: layer.gated_linear(x, w[:, :63]),
                lambda: layer.gated_linear(x, w, bias=torch.ones(8, device="cuda")), lambda: layer.gated_linear(x, w, activation="tanh"),
                lambda: layer.gated_linear(x.cpu(), w.cpu()), lambda: layer.gated_linear(x, w.t().contiguous().t()),
                lambda: layer.gated_linear(x.view(-1), w), lambda: layer.gated_linear_backward(z, x, w, z),
                lambda: layer.gated_linear_backward(y, x, w, y), lambda: layer.gated_linear_backward(y, x, w[:15], z)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(layer.LayerError):
        layer.gated_linear(x, w[:0])


def test_outputs_past_32_bits():
    """z and y past 2^31 values; all rows but a few are zero."""
    I, F = 16, 24
    T = (1 << 31) // F + 12345
    g = gen(9)
    at = torch.tensor([0, 1, 255, T // 2, T - 2, T - 1], device="cuda")
    x = torch.zeros(T, I, dtype=BF, device="cuda")
    x[at] = normal(g, 6, I, dtype=BF)
    w = normal(g, 2 * F, I, dtype=BF)
    y, z = layer.gated_linear_preact(x, w)
    want = x[at].double() @ w.double().t()
    off = sums(I, x[at].double().abs() @ w.double().abs().t()) + 4 * E * (want.abs() + 1)
    within(z[at], want, off + U[BF] * want.abs(), "z")
    check(y[at], want, off, "silu", BF)
    assert int((z.view(torch.int16) != 0).any(-1).sum()) == 6 and int((y.view(torch.int16) != 0).any(-1).sum()) <= 6
    # the gradients' u passes them too
    gy = torch.zeros(T, F, dtype=BF, device="cuda")
    gy[at] = normal(g, 6, F, dtype=BF)
    gx, gw, gb = layer.gated_linear_backward(gy, x, w, z)
    z64, g64 = z[at].double(), gy[at].double()
    a, s = act_ref(z64[:, :F], "silu")
    u = torch.cat([g64 * z64[:, F:] * s, g64 * a], 1)
    coarse = 1.1 * U[BF] * u.abs() + 2.0 ** -18 * (1 + z64.abs()) * g64.abs().repeat(1, 2) * (1 + z64.abs().amax())
    want = u @ w.double()
    within(gx[at], want, coarse @ w.double().abs() + sums(2 * F, u.abs() @ w.double().abs()) + U[BF] * want.abs(), "grad_x")
    assert int((gx.view(torch.int16) != 0).any(-1).sum()) == 6
    want = u.t() @ x[at].double()
    within(gw, want, coarse.t() @ x[at].double().abs() + sums(16, u.abs().t() @ x[at].double().abs()) + U[BF] * want.abs(), "grad_w")


def differences(f, args, h=1e-5):
    out = []
    for k, a in enumerate(args):
        d = torch.zeros_like(a)
        for i in range(a.numel()):
            v = [b.clone() for b in args]
            v[k].view(-1)[i] += h
            high = f(*v)
            v[k].view(-1)[i] -= 2 * h
            d.view(-1)[i] = (high - f(*v)) / (2 * h)
        out.append(d)
    return out


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gradient_against_differences(act):
    g = gen(22)
    F = 5
    x = normal(g, 3, 10, dtype=HF).requires_grad_()
    w = normal(g, 2 * F, 10, dtype=HF, spread=0.3).requires_grad_()
    b = normal(g, 2 * F).requires_grad_()
    c = normal(g, 3, F, dtype=HF)
    autograd.gated_linear(x, w, bias=b, activation=act).backward(c)

    def f(x64, w64, b64):
        z = x64 @ w64.t() + b64
        return (act_ref(z[:, :F], act)[0] * z[:, F:] * c.cpu().double()).sum()

    want = differences(f, [t.detach().cpu().double() for t in (x, w, b)])
    for got, ref in zip((x.grad, w.grad, b.grad), want):
        # z (both halves), u and the result are rounded to 11 bits each; |z| and |c| reach 4
        assert (got.cpu().double() - ref).abs().max() <= 2.0 ** -6 * (1 + ref.abs().max())


def test_autograd():
    g = gen(24)
    x = normal(g, 4, 3, 16, dtype=BF).requires_grad_()
    w, b = normal(g, 8, 16, dtype=BF).requires_grad_(), normal(g, 8).requires_grad_()
    y = autograd.gated_linear(x, w, bias=b)
    assert y.shape == (4, 3, 4)
    y.backward(torch.ones_like(y))
    z = layer.gated_linear_preact(x.detach().view(12, 16), w.detach(), bias=b.detach())[1]
    want = layer.gated_linear_backward(torch.ones(12, 4, dtype=BF, device="cuda"), x.detach().view(12, 16), w.detach(), z)
    assert torch.equal(x.grad.view(12, 16), want[0]) and torch.equal(w.grad, want[1]) and torch.equal(b.grad, want[2])
    with torch.no_grad():
        assert torch.equal(autograd.gated_linear(x, w, bias=b), y)
    # transposed and broadcast inputs are laid out first
    xt = normal(g, 16, 12, dtype=BF).t()
    assert torch.equal(autograd.gated_linear(xt, w), autograd.gated_linear(xt.contiguous(), w))
    xb = normal(g, 16, dtype=BF).expand(12, 16)
    assert torch.equal(autograd.gated_linear(xb, w), autograd.gated_linear(xb.contiguous(), w))
    loss = autograd.gated_linear(x, w).float().sum()
    grad, = torch.autograd.grad(loss, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        (loss + grad.float().pow(2).sum()).backward()


def test_weights_made_by_the_launch_before():
    """A few rows' product reads its weight ahead of the launch before it, which here writes that weight, over and over."""
    T, I, F = 8, 1024, 4096
    g = gen(91)
    x, a = normal(g, T, I, dtype=BF), normal(g, 2 * F, 256, dtype=BF)
    b = [normal(g, I, 256, dtype=BF, spread=2.0 ** -8) for _ in range(4)]
    want = []
    for k in range(4):
        w = layer.linear(a, b[k])
        torch.cuda.synchronize()
        want.append(layer.gated_linear(x, w).clone())
    assert not torch.equal(want[0], want[1])
    lib = layer.load()
    w, y = torch.empty(2 * F, I, dtype=BF, device="cuda"), [torch.empty(T, F, dtype=BF, device="cuda") for _ in range(40)]
    s = torch.cuda.current_stream().cuda_stream
    for i in range(40):
        assert lib.mhc_linear_fwd(a.data_ptr(), b[i % 4].data_ptr(), 0, 0, w.data_ptr(), 0, 0, 0, 2 * F, 256, I, 256, 256, I, 0, 0, s) == 0
        assert lib.mhc_gated_linear_fwd(x.data_ptr(), w.data_ptr(), 0, y[i].data_ptr(), 0, 0, 0, T, I, F, I, I, 2, 0, s) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(y[i], want[i % 4]) for i in range(40))
