"""The norm's ring kernels (many rows of more than 1024 values), whose blocks
take row after row through stages that bulk copies refill: against the
definitions in 64 bits, and byte for byte against the same rows in short
batches, which the row kernels take.

The sizes give a block more rows than its ring has stages.  Tolerances as in
test_layer_gpu.py: u = 2^-8 or 2^-11 of a rounded result, and 2^-24 of the sum
of magnitudes for each addition of a chain.
"""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, autograd, layer

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {BF: 2.0 ** -133, F16: 2.0 ** -24}
E = 2.0 ** -24
SHORT = 100     # rows of a call that the row kernels take: fewer than there are SMs


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()
    layer.wait_timeouts()
    yield
    assert layer.wait_timeouts() == 0


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((off - bound).max()):.3g} over"


def rows(g, T, H, dtype, pad, spread=1.0):
    """Random rows, `pad` values apart; what lies between must not be read."""
    t = torch.full((T, H + pad), float("nan"), device="cuda", dtype=dtype)
    t[:, :H] = (torch.randn(T, H, generator=g, device="cuda") * spread).to(dtype)
    return t[:, :H]


# Threads of a row, chunks of a thread and stages differ: 96 x 2, 128 x 2, 448 x 2, 512 x 2 (the widest form), 384 x 4, 512 x 4
FORWARD = [(24000, 1032), (15000, 2048), (6000, 7168), (5000, 8192), (4000, 12288), (2600, 16384)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("with_r", [False, True])
@pytest.mark.parametrize("T,H", FORWARD)
def test_forward(T, H, with_r, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    pad = 0 if dtype == BF else 16
    x, r = rows(g, T, H, dtype, pad, 3.0), rows(g, T, H, dtype, 2 * pad) if with_r else None
    w = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    odd = [17, T // 2, T - 1]          # NaN, infinity, zeros: in their rows alone
    x[17, 5], x[T // 2, H - 1] = float("nan"), float("inf")
    x[T - 1] = 0
    if with_r:
        r[T - 1] = 0
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[odd] = False
    s = x[keep].double() + (r[keep].double() if with_r else 0)
    rstd = 1 / torch.sqrt((s * s).mean(-1) + 1e-6)
    v = s * rstd[:, None] * w.double()

    y, total, got = layer.rms_norm(x, w, residual=r)
    within(got[keep], rstd, rstd * 64 * E, "rstd")
    within(y[keep], v, v.abs() * (U[dtype] + 80 * E) + TINY[dtype], "y")
    if with_r:
        within(total[keep], s, s.abs() * (U[dtype] + E) + TINY[dtype], "total")
    assert y[17].isnan().all() and y[T // 2, H - 1].isnan() and not y[T // 2, :H - 1].any() and not y[T - 1].any()
    outs = {None: (y, total, got)}

    for group in (0, 128):
        y8, scale, total8, got8 = layer.rms_norm_fp8(x, w, residual=r, group=group)
        assert same(total8.contiguous(), total.contiguous()) and same(got8, got)
        size, n = group or H, scale.shape[1]
        p = torch.zeros(v.shape[0], n * size, dtype=torch.float64, device="cuda")
        p[:, :H] = v
        q = torch.zeros_like(p)
        q[:, :H] = y8[keep].double()
        p, q = p.view(-1, n, size), q.view(-1, n, size)
        sc = p.abs().amax(-1).clamp(min=2.0 ** -60) / 448
        within(scale[keep], sc, sc * 90 * E, f"scale {group}")
        # 3 mantissa bits: half a unit is 2^-4 of the value, 2^-10 below the normal range
        within(q * scale[keep].double()[..., None], p, p.abs() * (2.0 ** -4 + 200 * E) + sc[..., None] * 2.0 ** -10, f"y8 {group}")
        assert scale[17].isnan().all() and (scale[T - 1] == 2.0 ** -60 / 448).all()
        outs[group] = (y8, scale, total8, got8)
        del p, q, sc
    del s, v

    # any split of the batch gives the same bytes: here in short calls, and again in one
    for group, whole in outs.items():
        def call(lo, hi):
            rr = None if r is None else r[lo:hi]
            return layer.rms_norm(x[lo:hi], w, residual=rr) if group is None else layer.rms_norm_fp8(x[lo:hi], w, residual=rr, group=group)
        for lo in [0, SHORT, T // 2 - 50, T - SHORT] + [T // 7 * i for i in range(1, 7)]:
            for a, b in zip(call(lo, lo + SHORT), whole):
                assert same(a.contiguous(), b[lo:lo + SHORT].contiguous()), (group, lo)
        for a, b in zip(call(0, T), whole):
            assert same(a.contiguous(), b.contiguous()), group


@pytest.mark.parametrize("H,lead", [(7168, 1), (2048, 3), (12288, 4)])
def test_rows_off_16_bytes_give_the_rings_bytes(H, lead):
    T = 3000
    g = torch.Generator(device="cuda").manual_seed(H)
    x = rows(g, T, H, BF, 0)
    w = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    off = torch.zeros(T, H + lead, dtype=BF, device="cuda")
    off[:, lead:] = x
    for a, b in zip(layer.rms_norm(off[:, lead:], w, residual=x), layer.rms_norm(x, w, residual=x)):
        assert same(a, b)
    y, _, rstd = layer.rms_norm(x, w)
    a, b = layer.rms_norm_backward(y, off[:, lead:], w, rstd), layer.rms_norm_backward(y, x, w, rstd)
    assert same(a[0], b[0])


BACKWARD = [(4000, 1032), (3000, 2048), (1000, 7168), (900, 8192), (700, 12288), (500, 16384)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("with_gt", [False, True])
@pytest.mark.parametrize("T,H", BACKWARD)
def test_backward(T, H, with_gt, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + H + 1)
    pad = 0 if dtype == BF else 8
    s, gy = rows(g, T, H, dtype, pad, 2.0), rows(g, T, H, dtype, 2 * pad)
    gt = rows(g, T, H, dtype, 0) if with_gt else None
    w = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    rstd = torch.rsqrt(s.float().square().mean(-1) + 1e-6)
    r64 = rstd.double()[:, None]
    n, u = s.double() * r64, gy.double() * w.double()
    more = gt.double() if with_gt else torch.zeros((), dtype=torch.float64, device="cuda")
    want = r64 * (u - n * (u * n).mean(-1, keepdim=True)) + more
    size = r64 * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True)) + more.abs()
    grad_x, grad_w = layer.rms_norm_backward(gy, s, w, rstd, grad_total=gt)
    within(grad_x, want, U[dtype] * want.abs() + 96 * E * size + TINY[dtype], "grad_x")
    # a block adds its rows (152 blocks or more), 128 groups of at most 5 blocks' sums are added, then 4 and 32 of them;
    # each term is a product of a rounded one
    terms = gy.double() * n
    within(grad_w, terms.sum(0), (-(-T // 152) + 5 + 2 + 5 + 4) * E * terms.abs().sum(0) + 1e-40, "grad_w")
    for lo in (0, 1, T // 3, T - SHORT):
        hi = lo + SHORT
        part, _ = layer.rms_norm_backward(gy[lo:hi], s[lo:hi], w, rstd[lo:hi], grad_total=None if gt is None else gt[lo:hi])
        assert same(part, grad_x[lo:hi].contiguous()), lo
    again = layer.rms_norm_backward(gy, s, w, rstd, grad_total=gt)
    assert same(again[0], grad_x) and same(again[1], grad_w)


def test_through_autograd():
    """The two-input form (total unused) and the three-input form give the operator's gradients."""
    T, H = 1000, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r, gy, gt = (rows(g, T, H, BF, 0) for _ in range(4))
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).requires_grad_()
    x.requires_grad_(), r.requires_grad_()
    for used in (False, True):
        y, total = autograd.rms_norm(x, w, residual=r)
        got = torch.autograd.grad([y, total][:1 + used], [x, w, r], [gy, gt][:1 + used])
        _, s, rstd = layer.rms_norm(x.detach(), w.detach(), residual=r.detach())
        want = layer.rms_norm_backward(gy, s, w.detach(), rstd, grad_total=gt if used else None)
        assert same(got[0], want[0]) and same(got[1], want[1]) and same(got[2], want[0])


def test_no_wait_runs_out():
    assert layer.wait_timeouts() == 0
    for T, H in ((1400, 7168), (3000, 1280), (700, 12288)):
        x = torch.ones(T, H, device="cuda", dtype=BF)
        w = torch.ones(H, device="cuda")
        y, total, rstd = layer.rms_norm(x, w, residual=x)
        layer.rms_norm_fp8(x, w, residual=x, group=128)
        layer.rms_norm_backward(y, total, w, rstd, grad_total=y)
    assert layer.wait_timeouts() == 0
