"""The product where its output side passes 32-bit offsets: y, its
pre-activation, the residual and the gradients' u past 2^31 values (2^32
bytes).  All rows but a few are zero, so that the sums have few terms."""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, layer

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -8
E23, E24 = 2.0 ** -23, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()
    yield
    torch.cuda.empty_cache()
    assert layer.wait_timeouts() == 0


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), f"{what}: worst {float((off - bound).max()):.3g} over"


# narrow rows (a tile of columns that is not full) and wide ones (many tiles, parts of K summed apart)
SIZES = [((1 << 31) // 24 + 12345, 16, 24), ((1 << 31) // 7168 + 333, 2048, 7168)]


@pytest.mark.parametrize("T,I,O", SIZES)
def test_outputs(T, I, O):
    assert T * O > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(O)
    at = torch.tensor([0, 1, 255, T // 2, T - 2, T - 1], device="cuda")
    x = torch.zeros(T, I, dtype=BF, device="cuda")
    x[at] = torch.randn(6, I, generator=g, device="cuda").to(BF)
    w = (torch.randn(O, I, generator=g, device="cuda") * I ** -0.5).to(BF)
    r = torch.zeros(T, O, dtype=BF, device="cuda")
    r[at] = torch.randn(6, O, generator=g, device="cuda").to(BF)
    y, z = layer.linear_preact(x, w, activation="relu", residual=r)
    want_z = x[at].double() @ w.double().t()
    want = want_z.clamp(min=0) + r[at].double()
    # one truncating addition per 16 products and the products' own alignment, then the rounding
    sums = (2 * -(-I // 16) + 32) * E23 * (x[at].double().abs() @ w.double().abs().t())
    within(z[at], want_z, 1.1 * sums + (U + E24) * want_z.abs(), "z")
    within(y[at], want, 1.1 * sums + (U + E24) * want.abs(), "y")
    for t in (y, z):      # nothing of any other row is written
        assert int((t.view(torch.int16) != 0).any(-1).sum()) == 6


def test_gradients():
    T, I, O = SIZES[0]
    g = torch.Generator(device="cuda").manual_seed(5)
    at = torch.tensor([0, 77, T // 2, T - 2, T - 1], device="cuda")
    x = torch.zeros(T, I, dtype=BF, device="cuda")
    gy, z = torch.zeros(T, O, dtype=BF, device="cuda"), torch.zeros(T, O, dtype=BF, device="cuda")
    for t in (x, gy, z):
        t[at] = torch.randn(5, t.shape[1], generator=g, device="cuda").to(BF)
    w = torch.randn(O, I, generator=g, device="cuda").to(BF)
    gx, gw, gb = layer.linear_backward(gy, x, w, z=z, activation="silu")
    z64 = z[at].double()
    p = torch.sigmoid(z64)
    slope = p * (1 + z64 * (1 - p))
    u = gy[at].double() * slope
    # its slope is within 2^-20; the products read it rounded to 8 bits, grad_b does not
    exact = gy[at].double().abs() * 2.0 ** -20 * (1 + z64.abs())
    off = exact + 1.01 * U * u.abs()
    want = u @ w.double()
    within(gx[at], want, off @ w.double().abs() + 64 * E23 * (u.abs() @ w.double().abs()) + U * want.abs(), "grad_x")
    assert int((gx.view(torch.int16) != 0).any(-1).sum()) == 5
    want = u.t() @ x[at].double()
    within(gw, want, off.t() @ x[at].double().abs() + 64 * E23 * (u.abs().t() @ x[at].double().abs()) + U * want.abs(), "grad_w")
    within(gb, u.sum(0), exact.sum(0) + 16 * E24 * u.abs().sum(0), "grad_b")
