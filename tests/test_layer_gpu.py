"""The layer operators (RMS norm, matrix product, rotary positions) on a GPU
against their definitions in 64 bits.

Tolerances follow from the number formats: a result rounded once to a storage
type of significand p bits is off by at most 2^-p of itself (u below: 2^-8
allows for BF16's 8 bits, 2^-11 for binary16's 11; half of that for rounding to
nearest is the actual bound, the other half covers FP32 results next to a
rounding boundary), and an FP32 sum of n terms in a chain of at most c
additions by c 2^-24 of the sum of the terms' magnitudes (2^-23 for sums inside
the tensor cores, which may truncate).
"""

import math

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, autograd, layer

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}   # spacing of the smallest values
E = 2.0 ** -24
BOTH = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    layer.load()
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
    """The same values in rows of a wider buffer."""
    T, H = t.shape
    b = torch.full((T, lead + H + extra), float("nan"), device="cuda").to(t.dtype)
    b[:, lead:lead + H] = t
    return b[:, lead:lead + H]


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def norm_ref(x, r, w, eps):
    s = x.double() + (0 if r is None else r.double())
    rstd = 1 / torch.sqrt((s * s).mean(-1) + eps)
    return s, rstd, s * rstd[:, None] * w.double()


NORM_SIZES = [(1, 7168), (5, 8), (3, 1), (7, 127), (33, 128), (9, 256), (4, 504), (6, 1024), (5, 1025), (2, 1032),
              (17, 1279), (3, 4097), (129, 2048), (2, 8192), (1, 32768), (2, 32767), (700, 640)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("with_r", [False, True])
def test_norm_forward(T, H, with_r, dtype):
    g = gen(T * 100003 + H)
    x = normal(g, T, H, dtype=dtype, spread=3.0)
    r = normal(g, T, H, dtype=dtype) if with_r else None
    w = 1 + normal(g, H, spread=0.3)
    s, rstd, v = norm_ref(x, r, w, 1e-5)
    y, total, got_rstd = layer.rms_norm(x, w, residual=r, eps=1e-5)
    within(got_rstd, rstd, rstd * 64 * E, "rstd")
    within(y, v, v.abs() * (U[dtype] + 80 * E) + TINY[dtype], "y")
    if with_r:
        within(total, s, s.abs() * (U[dtype] + E) + TINY[dtype], "total")
    else:
        assert total is x


def check_fp8(v, y8, scale, group):
    T, H = v.shape
    size = group or H
    q = y8.double()
    for i in range(scale.shape[1]):
        part = v[:, i * size:(i + 1) * size]
        sc = part.abs().amax(-1).clamp(min=2.0 ** -60) / 448
        within(scale[:, i], sc, sc * 90 * E, f"scale {i}")
        # 3 mantissa bits: half a unit is 2^-4 of the value, 2^-10 below the normal range
        back = q[:, i * size:(i + 1) * size] * scale[:, i:i + 1].double()
        within(back, part, part.abs() * (2.0 ** -4 + 200 * E) + sc[:, None] * 2.0 ** -10, f"y8 {i}")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,H", [(1, 7168), (5, 8), (3, 127), (4, 128), (9, 136), (7, 1000), (2, 1023), (33, 1279),
                                 (3, 4097), (65, 2048), (1, 32767)])
def test_norm_fp8(T, H, group, dtype):
    g = gen(T * 100003 + H + group)
    x = normal(g, T, H, dtype=dtype, spread=2.0)
    r = normal(g, T, H, dtype=dtype)
    w = 1 + normal(g, H, spread=0.3)
    s, rstd, v = norm_ref(x, r, w, 1e-6)
    y8, scale, total, got_rstd = layer.rms_norm_fp8(x, w, residual=r, group=group)
    assert y8.dtype == torch.float8_e4m3fn and scale.shape == (T, 1 if group == 0 else -(-H // 128))
    check_fp8(v, y8, scale, group)
    within(total, s, s.abs() * (U[dtype] + E) + TINY[dtype], "total")
    # the 16-bit output's rstd and total have the same bits
    _, total2, rstd2 = layer.rms_norm(x, w, residual=r)
    assert torch.equal(total, total2) and torch.equal(got_rstd, rstd2)


@pytest.mark.parametrize("H", [512, 7168, 1279])
def test_norm_special_rows(H):
    x = torch.zeros(6, H, device="cuda", dtype=torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 3e38            # the sum of squares overflows: rstd 0
    x[4] = 1e-38           # and underflows: eps alone
    x[5] = 1
    w = torch.ones(H, device="cuda")
    y, _, rstd = layer.rms_norm(x, w, eps=1e-6)
    assert torch.equal(y[0], torch.zeros_like(y[0])) and rstd[0].item() == pytest.approx(1e3, rel=1e-6)
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 5]) and (y[2, :5] == 0).all()
    assert rstd[3] == 0 and (y[3] == 0).all()
    assert rstd[4].item() == pytest.approx(1e3, rel=1e-6)
    assert (y[5] == 1).all()
    for group in (0, 128):
        q, scale, _, _ = layer.rms_norm_fp8(x, w, eps=1e-6, group=group)
        q = q.float()
        assert (q[0] == 0).all() and torch.equal(scale[0], torch.full_like(scale[0], 2.0 ** -60 / 448))
        assert torch.isnan(q[1]).all() and torch.isnan(scale[1]).all()
        assert torch.isnan(scale[2, 0])
        assert (q[5] == 448).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,H", [(1, 7168), (5, 8), (3, 1), (7, 127), (40, 128), (9, 1000), (6, 1024), (5, 1025),
                                 (17, 1279), (3, 4097), (650, 2048), (1300, 256), (2, 8192), (1, 32768), (2, 32767),
                                 (321, 1279)])
def test_norm_backward(T, H, dtype):
    g = gen(T * 100003 + H + 7)
    s = normal(g, T, H, dtype=dtype, spread=2.0)
    gy = normal(g, T, H, dtype=dtype)
    gt = normal(g, T, H, dtype=dtype) if T % 2 else None
    w = 1 + normal(g, H, spread=0.3)
    rstd = torch.rsqrt(s.float().square().mean(-1) + 1e-6)
    r64 = rstd.double()[:, None]
    n = s.double() * r64
    u = gy.double() * w.double()
    m = (u * n).mean(-1, keepdim=True)
    want = r64 * (u - n * m) + (0 if gt is None else gt.double())
    grad_x, grad_w = layer.rms_norm_backward(gy, s, w, rstd, grad_total=gt)
    size = r64 * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True)) + (0 if gt is None else gt.double().abs())
    within(grad_x, want, U[dtype] * want.abs() + 96 * E * size + TINY[dtype], "grad_x")
    chain = math.ceil(T / 300) + 64
    within(grad_w, (gy.double() * n).sum(0), (chain + 8) * E * (gy.double() * n).abs().sum(0) + 1e-40, "grad_w")


@pytest.mark.parametrize("H", [640, 7168])
def test_norm_alignment_and_stride(H):
    """Rows off 16 bytes and strided rows give the same bytes as dense aligned ones."""
    g = gen(H)
    T = 11
    x, r, gy = (normal(g, T, H, dtype=torch.bfloat16) for _ in range(3))
    w = 1 + normal(g, H, spread=0.3)
    want = layer.rms_norm(x, w, residual=r)
    want8 = layer.rms_norm_fp8(x, w, residual=r, group=128)
    grad, _ = layer.rms_norm_backward(gy, want[1], w, want[2])
    for lead, extra in ((0, 8), (1, 0), (8, 16), (3, 2)):
        xs, rs = strided(x, extra, lead), strided(r, extra, lead)
        got = layer.rms_norm(xs, w, residual=rs)
        got8 = layer.rms_norm_fp8(xs, w, residual=rs, group=128)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, b in zip(got8, want8):
            assert torch.equal(a.float(), b.float())
        got_grad, _ = layer.rms_norm_backward(strided(gy, extra, lead), strided(want[1], extra, lead), w, want[2])
        assert torch.equal(got_grad, grad)


@pytest.mark.parametrize("H", [200, 1279, 7168])
def test_norm_split_and_repeat(H):
    g = gen(H + 1)
    x, r = (normal(g, 67, H, dtype=torch.float16) for _ in range(2))
    w = 1 + normal(g, H, spread=0.3)
    whole = layer.rms_norm_fp8(x, w, residual=r, group=128)
    for _ in range(5):
        again = layer.rms_norm_fp8(x, w, residual=r, group=128)
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(whole, again))
    for i in (0, 13, 66):
        one = layer.rms_norm_fp8(x[i:i + 1], w, residual=r[i:i + 1], group=128)
        assert all(torch.equal(a[0].float(), b[i].float()) for a, b in zip(one, whole))


# ---------------------------------------------------------------------------
# matrix product
# ---------------------------------------------------------------------------

def act_ref(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    return z


def slope_ref(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def sum_bound(K, size):
    """Of a tensor-core sum over K: one truncating addition per 16 products, the products' own alignment, the parts."""
    return (2 * math.ceil(K / 16) + 32) * 2.0 ** -23 * size


def linear_case(T, I, O, dtype, act, bias, residual, seed=0, fp8=False):
    g = gen(T + 7 * I + 13 * O + seed)
    x, w = normal(g, T, I), normal(g, O, I, spread=I ** -0.5)
    sx = sw = None
    if fp8:
        sx, sw = x.abs().amax(-1) / 448, w.abs().amax(-1) / 448
        x, w = ((a / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for a, s in ((x, sx), (w, sw)))
    else:
        x, w = x.to(dtype), w.to(dtype)
    b = normal(g, O) if bias else None
    r = normal(g, T, O, dtype=dtype) if residual else None
    x64, w64 = x.double(), w.double()
    if fp8:
        x64, w64 = x64 * sx.double()[:, None], w64 * sw.double()[:, None]
    z = x64 @ w64.t() + (0 if b is None else b.double())
    size = x64.abs() @ w64.abs().t()
    y = act_ref(z, act) + (0 if r is None else r.double())
    bound = 1.2 * sum_bound(I, size) + U[dtype] * y.abs() + 64 * E * (z.abs() + 1 + y.abs()) + TINY[dtype]
    return x, sx, w, sw, b, r, z, y, bound, size


LINEAR_SIZES = [(1, 7168, 1024), (1, 64, 8), (1, 1, 1), (2, 8, 24), (3, 100, 130), (16, 128, 128), (17, 256, 129),
                (64, 520, 300), (129, 1279, 513), (200, 64, 2048), (256, 192, 256), (257, 320, 40), (300, 1024, 520),
                (513, 72, 1000), (1000, 640, 264), (2049, 328, 2600)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,I,O", LINEAR_SIZES)
def test_linear(T, I, O, dtype):
    for act, bias, residual in (("none", False, False), ("silu", True, True)):
        x, _, w, _, b, r, z, y, bound, size = linear_case(T, I, O, dtype, act, bias, residual)
        got = layer.linear(x, w, bias=b, activation=act, residual=r)
        within(got, y, bound, f"y {act}")
    got, got_z = layer.linear_preact(x, w, bias=b, activation=act, residual=r)
    within(got, y, bound, "y")
    within(got_z, z, sum_bound(I, size) + (U[dtype] + 4 * E) * z.abs() + TINY[dtype] + 4 * E, "z")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True)])
@pytest.mark.parametrize("T", [5, 600])
def test_linear_epilogues(T, act, bias, residual):
    x, _, w, _, b, r, z, y, bound, _ = linear_case(T, 264, 2300, torch.bfloat16, act, bias, residual)
    within(layer.linear(x, w, bias=b, activation=act, residual=r), y, bound, "y")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,I,O", [(1, 7168, 512), (1, 16, 8), (3, 17, 5), (64, 512, 300), (129, 1280, 513),
                                   (256, 144, 128), (700, 1000, 260), (2049, 336, 2600)])
def test_linear_fp8(T, I, O, dtype):
    x, sx, w, sw, b, r, z, y, bound, _ = linear_case(T, I, O, dtype, "gelu", True, True, fp8=True)
    within(layer.linear_fp8(x, sx, w, sw, bias=b, activation="gelu", residual=r, dtype=dtype), y, bound, "y")


def test_norm_into_linear_fp8():
    """The norm's 8-bit output and its [T,1] scales feed the product as they are."""
    g = gen(5)
    x = normal(g, 33, 1024, dtype=torch.bfloat16)
    wn = 1 + normal(g, 1024, spread=0.2)
    w = normal(g, 256, 1024, spread=1 / 32)
    sw = w.abs().amax(-1) / 448
    w8 = (w / sw[:, None]).to(torch.float8_e4m3fn)
    y8, scale, _, _ = layer.rms_norm_fp8(x, wn)
    got = layer.linear_fp8(y8, scale, w8, sw)
    a, b = y8.double() * scale.double(), w8.double() * sw.double()[:, None]
    want = a @ b.t()
    within(got, want, sum_bound(1024, a.abs() @ b.abs().t()) + U[torch.bfloat16] * want.abs() + 8 * E, "y")


@pytest.mark.parametrize("lead,extra", [(0, 8), (8, 8), (1, 0), (0, 1), (3, 5)])
def test_linear_strides(lead, extra):
    """Strided and misaligned operands give the same bytes as dense ones."""
    x, _, w, _, b, r, *_ = linear_case(37, 200, 333, torch.bfloat16, "silu", True, True)
    want = layer.linear(x, w, bias=b, activation="silu", residual=r)
    got = layer.linear(strided(x, extra, lead), strided(w, extra, lead), bias=b, activation="silu",
                       residual=strided(r, extra, lead))
    assert torch.equal(got, want)


@pytest.mark.parametrize("I,O", [(7168, 2048), (4096, 7168), (1024, 1024), (1279, 300), (512, 24)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_rows_do_not_depend_on_the_batch(I, O, fp8):
    """A token's y and grad_x have the same bits alone, in a decode batch and in a prefill."""
    if fp8:
        I = I // 16 * 16
    T = 1500
    x, sx, w, sw, b, r, *_ = linear_case(T, I, O, torch.bfloat16, "silu", True, True, fp8=fp8)

    def run(lo, hi):
        if fp8:
            return layer.linear_fp8(x[lo:hi], sx[lo:hi], w, sw, bias=b, activation="silu", residual=r[lo:hi])
        return layer.linear(x[lo:hi], w, bias=b, activation="silu", residual=r[lo:hi])

    whole = run(0, T)
    assert torch.equal(run(0, T), whole)
    for lo, hi in ((0, 1), (777, 778), (1499, 1500), (3, 40), (100, 229), (640, 940), (0, 700)):
        assert torch.equal(run(lo, hi), whole[lo:hi]), (lo, hi)
    if not fp8:
        gy = r.contiguous()
        gx = layer.linear_backward(gy, x, w, bias=False, want=(True, False))[0]
        for lo, hi in ((0, 1), (3, 40), (640, 940)):
            part = layer.linear_backward(gy[lo:hi].contiguous(), x[lo:hi].contiguous(), w, bias=False, want=(True, False))[0]
            assert torch.equal(part, gx[lo:hi]), (lo, hi)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("T,I,O", [(1, 64, 8), (3, 100, 130), (65, 256, 128), (129, 1279, 513), (300, 520, 24),
                                   (2049, 328, 2600), (1, 1, 1), (700, 2300, 72)])
def test_linear_backward(T, I, O, act, dtype):
    g = gen(T + I + O)
    x, w = normal(g, T, I, dtype=dtype), normal(g, O, I, dtype=dtype, spread=O ** -0.5)
    z, gy = normal(g, T, O, dtype=dtype), normal(g, T, O, dtype=dtype)
    u = gy.double() * slope_ref(z.double(), act)
    got = layer.linear_backward(gy, x, w, z=None if act == "none" else z, activation=act)
    # cvt(u) is off by u itself, one more rounding of the result
    ux = 0 if act == "none" else 1.01 * U[dtype]
    slope_err = 0 if act == "none" else 2.0 ** -20 * gy.double().abs() * (1 + z.double().abs())
    size = u.abs() @ w.double().abs()
    want = u @ w.double()
    small = (slope_err + TINY[dtype]) if act != "none" else torch.zeros_like(u)
    within(got[0], want, sum_bound(O, size) + ux * size + small @ w.double().abs() + U[dtype] * want.abs() + TINY[dtype],
           "grad_x")
    size = u.abs().t() @ x.double().abs()
    want = u.t() @ x.double()
    within(got[1], want, sum_bound(T, size) + ux * size + small.t() @ x.double().abs() + U[dtype] * want.abs() + TINY[dtype],
           "grad_w")
    chain = math.ceil(T / 64) + 72
    within(got[2], u.sum(0), chain * E * u.abs().sum(0) + (slope_err.sum(0) if act != "none" else 0) + 1e-30, "grad_b")
    # each gradient alone has the same bits
    one = layer.linear_backward(gy, x, w, z=z, activation=act, bias=False, want=(True, False))
    assert one[1] is None and one[2] is None and torch.equal(one[0], got[0])
    one = layer.linear_backward(gy, x, w, z=z, activation=act, bias=False, want=(False, True))
    assert one[0] is None and torch.equal(one[1], got[1])
    one = layer.linear_backward(gy, x, w, z=z, activation=act, want=(False, False))
    assert torch.equal(one[2], got[2])


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("T,D", [(40, 328), (700, 520), (2049, 1032), (700, 1023)])
def test_linear_backward_calls_in_a_row(T, D, act):
    """The kernels of a call overlap: grad_x read, and freed memory taken, by the call right after it."""
    g = gen(T + D)
    w = [normal(g, D, D, dtype=torch.bfloat16, spread=D ** -0.5) for _ in range(6)]
    x, z, first = (normal(g, T, D, dtype=torch.bfloat16) for _ in range(3))

    def chain(wait):
        gy, out = first, []
        for weight in w:
            got = layer.linear_backward(gy, x, weight, z=None if act == "none" else z, activation=act)
            wait()
            out += got
            gy = got[0]
        return out

    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_linear_masked_values():
    """NaN and infinities stay in the rows that hold them, also next to ragged edges."""
    x, _, w, _, _, _, _, y, bound, _ = linear_case(70, 100, 150, torch.bfloat16, "none", False, False)
    x[3, 7] = float("nan")
    x[69, 99] = float("inf")
    got = layer.linear(x, w)
    keep = [i for i in range(70) if i not in (3, 69)]
    within(got[keep], y[keep], bound[keep], "other rows")
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[69]).any()


def test_linear_long_rows_past_32_bits():
    """Offsets past 2^31 values in an operand and past 2^32 bytes in the output."""
    O, I = 24, 64
    T = (1 << 31) // 24 // 2 + 12345          # y: 2^30 values
    stride = 64
    g = gen(9)
    x = torch.zeros(T, stride, dtype=torch.bfloat16, device="cuda")   # 2.9e9 values
    rows = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    x[rows] = normal(g, 5, stride, dtype=torch.bfloat16)
    w = normal(g, O, I, dtype=torch.bfloat16)
    got = layer.linear(x, w)
    want = x[rows].double() @ w.double().t()
    within(got[rows], want, sum_bound(I, x[rows].double().abs() @ w.double().abs().t()) + U[torch.bfloat16] * want.abs(), "y")
    assert int((got != 0).any(-1).sum()) == 5


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rotary_ref(x, pos, f, interleaved, scale, inverse):
    R = 2 * f.numel()
    angle = pos.double()[:, None] * f.double()
    c, s = (torch.cos(angle) * scale)[:, None], (torch.sin(angle) * scale * (-1 if inverse else 1))[:, None]
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    first = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., first[0]], y[..., first[1]] = a * c - b * s, b * c + a * s
    size[..., first[0]] = size[..., first[1]] = scale * (a.abs() + b.abs())
    return y, size


def check_rotary(got, x, pos, f, interleaved, scale, inverse):
    y, size = rotary_ref(x, pos, f, interleaved, scale, inverse)
    # the angle to 2^-20, its sine and cosine and the products to a few FP32 units
    within(got, y, U[x.dtype] * y.abs() + 2.0 ** -19 * size + TINY[x.dtype], "rotary")
    assert torch.equal(got[..., 2 * f.numel():], x[..., 2 * f.numel():])


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,D,R", [(1, 1, 64, 64), (3, 5, 128, 128), (7, 8, 128, 64), (2, 40, 192, 64),
                                         (5, 3, 80, 20), (4, 9, 96, 24), (6, 2, 7, 2), (129, 16, 256, 256), (9, 4, 64, 0),
                                         (2, 1, 6, 6), (1000, 12, 128, 128)])
def test_rotary(T, heads, D, R, interleaved, dtype):
    g = gen(T + heads * 31 + D + R)
    x = normal(g, T, heads, D, dtype=dtype)
    pos = torch.randint(0, 131072, (T,), generator=g, device="cuda")
    f = layer.rotary_frequencies(R) if R else torch.empty(0, device="cuda")
    for inverse in (False, True):
        got = layer.rotary(x, pos, f, interleaved=interleaved, scale=1.25, inverse=inverse)
        check_rotary(got, x, pos, f, interleaved, 1.25, inverse)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_long_positions(interleaved):
    g = gen(3)
    pos = torch.tensor([0, 1, -5, 1 << 20, (1 << 24) + 1, 12345678], device="cuda")
    x = normal(g, 6, 2, 64, dtype=torch.float16)
    f = layer.rotary_frequencies(64)
    check_rotary(layer.rotary(x, pos, f, interleaved=interleaved), x, pos, f, interleaved, 1.0, False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lead", [0, 1, 2, 4, 8])
def test_rotary_strides_and_in_place(lead, interleaved):
    """Heads inside wider rows at every alignment, out of place, into strided rows and in place."""
    g = gen(lead)
    T, heads, D = 13, 6, 64
    rows = normal(g, T, lead + (heads + 2) * D, dtype=torch.bfloat16)
    x = rows[:, lead:lead + heads * D].unflatten(1, (heads, D))
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda")
    f = layer.rotary_frequencies(48, scaling="yarn", factor=4.0)
    want = layer.rotary(x.contiguous(), pos, f, interleaved=interleaved)
    check_rotary(want, x, pos, f, interleaved, 1.0, False)
    assert torch.equal(layer.rotary(x, pos, f, interleaved=interleaved), want)
    # heads outermost in memory
    other = torch.zeros(heads, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    if lead == 0:
        with pytest.raises(layer.LayerError):     # a token's heads must not interleave with the next token's
            layer.rotary(x, pos, f, interleaved=interleaved, out=other)
    before = rows.clone()
    assert layer.rotary(x, pos, f, interleaved=interleaved, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(x, want)
    before[:, lead:lead + heads * D] = want.flatten(1)
    assert torch.equal(rows, before)


def test_rotary_frequency_tables():
    full = layer.rotary_frequencies(128, device="cpu").double()
    assert torch.allclose(full, 10000.0 ** (-torch.arange(0, 128, 2).double() / 128), rtol=2.0 ** -23)
    assert torch.equal(layer.rotary_frequencies(128, scaling="linear", factor=8.0, device="cpu").double(), full / 8)
    ntk = layer.rotary_frequencies(128, scaling="ntk", factor=8.0, device="cpu").double()
    assert ntk[0] == 1 and abs(ntk[-1] / (full[-1] / 8) - 1) < 1e-6
    yarn = layer.rotary_frequencies(128, scaling="yarn", factor=8.0, trained=4096, device="cpu").double()
    assert yarn[0] == full[0] and abs(yarn[-1] / (full[-1] / 8) - 1) < 1e-6 and (yarn <= full).all()


# ---------------------------------------------------------------------------
# gradients through autograd, against differences of the 64-bit definitions
# ---------------------------------------------------------------------------

def differences(f, args, h=1e-5):
    """Central differences of the scalar f in every entry of every argument (64 bits)."""
    out = []
    for k, a in enumerate(args):
        d = torch.zeros_like(a)
        flat = d.view(-1)
        for i in range(a.numel()):
            v = [b.clone() for b in args]
            v[k].view(-1)[i] += h
            up = f(*v)
            v[k].view(-1)[i] -= 2 * h
            flat[i] = (up - f(*v)) / (2 * h)
        out.append(d)
    return out


def test_norm_gradient_against_differences():
    g = gen(21)
    x, r = (normal(g, 2, 12, dtype=torch.float16).requires_grad_() for _ in range(2))
    w = (1 + normal(g, 12, spread=0.3)).requires_grad_()
    cy, ct = normal(g, 2, 12, dtype=torch.float16), normal(g, 2, 12, dtype=torch.float16)
    y, total = autograd.rms_norm(x, w, residual=r)
    torch.autograd.backward([y, total], [cy, ct])

    def f(x64, r64, w64):
        s, _, v = norm_ref(x64, r64, w64, 1e-6)
        return (v * cy.cpu().double()).sum() + (s * ct.cpu().double()).sum()

    want = differences(f, [t.detach().cpu().double() for t in (x, r, w)])
    for got, ref in zip((x.grad, r.grad, w.grad), want):
        # total's rounding (2^-11) moves n, and so the gradient, by about as much
        assert (got.cpu().double() - ref).abs().max() <= 2.0 ** -9 * (1 + ref.abs().max())


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_linear_gradient_against_differences(act):
    g = gen(22)
    x = normal(g, 3, 10, dtype=torch.float16).requires_grad_()
    w = normal(g, 5, 10, dtype=torch.float16, spread=0.3).requires_grad_()
    b = normal(g, 5).requires_grad_()
    r = normal(g, 3, 5, dtype=torch.float16).requires_grad_()
    c = normal(g, 3, 5, dtype=torch.float16)
    autograd.linear(x, w, bias=b, activation=act, residual=r).backward(c)

    def f(x64, w64, b64, r64):
        return ((act_ref(x64 @ w64.t() + b64, act) + r64) * c.cpu().double()).sum()

    want = differences(f, [t.detach().cpu().double() for t in (x, w, b, r)])
    for got, ref in zip((x.grad, w.grad, b.grad, r.grad), want):
        # z, u and the result are rounded to 11 bits each
        assert (got.cpu().double() - ref).abs().max() <= 2.0 ** -8 * (1 + ref.abs().max())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient_against_differences(interleaved):
    g = gen(23)
    x = normal(g, 2, 2, 12, dtype=torch.float16).requires_grad_()
    pos = torch.tensor([3, 1000], device="cuda")
    f = layer.rotary_frequencies(8)
    c = normal(g, 2, 2, 12, dtype=torch.float16)
    autograd.rotary(x, pos, f, interleaved=interleaved, scale=1.5).backward(c)
    want = differences(lambda v: (rotary_ref(v, pos.cpu(), f.cpu(), interleaved, 1.5, False)[0] * c.cpu().double()).sum(),
                       [x.detach().cpu().double()])[0]
    assert (x.grad.cpu().double() - want).abs().max() <= 2.0 ** -10 * (1 + want.abs().max())


def test_autograd_without_the_optional_parts():
    g = gen(24)
    x = normal(g, 4, 3, 16, dtype=torch.bfloat16).requires_grad_()      # leading batch shape
    w = torch.ones(16, device="cuda")
    y, total = autograd.rms_norm(x, w)
    assert y.shape == x.shape and torch.equal(total, x)
    wl = normal(g, 8, 16, dtype=torch.bfloat16).requires_grad_()
    out = autograd.linear(y, wl)
    assert out.shape == (4, 3, 8)
    out.backward(torch.ones_like(out))
    assert x.grad.shape == x.shape and wl.grad.shape == wl.shape and torch.isfinite(x.grad.float()).all()


# ---------------------------------------------------------------------------
# streams, empty calls, refusals
# ---------------------------------------------------------------------------

def test_other_stream():
    g = gen(31)
    x, w = normal(g, 300, 512, dtype=torch.bfloat16), normal(g, 700, 512, dtype=torch.bfloat16)
    wn = torch.ones(512, device="cuda")
    want = layer.linear(layer.rms_norm(x, wn)[0], w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer.linear(layer.rms_norm(x, wn)[0], w)
    side.synchronize()
    assert torch.equal(got, want)
    got = layer.linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, layer.linear(x, w))


def test_in_a_graph():
    g = gen(32)
    x, w = normal(g, 40, 512, dtype=torch.bfloat16), normal(g, 700, 512, dtype=torch.bfloat16)
    wn = torch.ones(512, device="cuda")
    want = layer.linear(layer.rms_norm(x, wn)[0], w, activation="silu")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.linear(layer.rms_norm(x, wn)[0], w, activation="silu")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_no_tokens():
    dev = "cuda"
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    y, total, rstd = layer.rms_norm(x, w, residual=x)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    grad_x, grad_w = layer.rms_norm_backward(x, x, w, rstd)
    assert grad_x.shape == (0, 64) and torch.equal(grad_w, torch.zeros(64, device=dev))
    wl = torch.ones(8, 64, dtype=torch.bfloat16, device=dev)
    assert layer.linear(x, wl).shape == (0, 8)
    gx, gw, gb = layer.linear_backward(torch.empty(0, 8, dtype=torch.bfloat16, device=dev), x, wl)
    assert gx.shape == (0, 64) and (gw == 0).all() and (gb == 0).all()
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=dev)
    assert layer.rotary(q, torch.empty(0, dtype=torch.int64, device=dev), layer.rotary_frequencies(64)).shape == q.shape


def test_refusals():
    dev = "cuda"
    x = torch.ones(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    wl = torch.ones(8, 64, dtype=torch.bfloat16, device=dev)
    f = layer.rotary_frequencies(64)
    pos = torch.zeros(4, dtype=torch.int64, device=dev)
    q = x.view(4, 1, 64)
    for bad in (lambda: layer.rms_norm(x.float(), w), lambda: layer.rms_norm(x, w.bfloat16()),
                lambda: layer.rms_norm(x, w, residual=x.half()), lambda: layer.linear(x, wl.half()),
                lambda: layer.linear(x, wl, bias=torch.ones(8, device=dev, dtype=torch.bfloat16)),
                lambda: layer.linear_fp8(x, w, wl, w), lambda: layer.rotary(q.float(), pos, f),
                lambda: layer.rotary(q, pos.int(), f), lambda: layer.rms_norm(None, w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: layer.rms_norm(x, w[:63]), lambda: layer.rms_norm(x.view(-1), w),
                lambda: layer.rms_norm(x.cpu(), w.cpu()), lambda: layer.rms_norm(x.t(), torch.ones(4, device=dev)),
                lambda: layer.rms_norm(x[:1].expand(4, 64), w), lambda: layer.linear(x, wl[:, :63]),
                lambda: layer.linear(x, wl, activation="tanh"), lambda: layer.linear(x, wl, residual=x),
                lambda: layer.linear_backward(torch.ones(4, 8, dtype=torch.bfloat16, device=dev), x, wl, activation="silu"),
                lambda: layer.rotary(q, pos[:3], f), lambda: layer.rotary(q, pos, f.view(1, -1)),
                lambda: layer.rotary_frequencies(63), lambda: layer.rotary_frequencies(64, scaling="other")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: layer.rms_norm(torch.ones(1, 32776, dtype=torch.bfloat16, device=dev), torch.ones(32776, device=dev)),
                lambda: layer.rms_norm_fp8(x, w, group=64), lambda: layer.rotary(q, pos, layer.rotary_frequencies(66)),
                lambda: layer.rotary(x.view(4, 1, 64), pos, f, out=x.view(-1)[:1].expand(4, 1, 64).contiguous().as_strided((4, 1, 64), (0, 64, 1)))):
        with pytest.raises(layer.LayerError):
            bad()


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------

def test_norm_past_32_bits():
    T, H = 300000, 7168                                       # 2.15e9 values
    g = gen(41)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, T // 2, T - 1], device="cuda")
    x[rows] = normal(g, 3, H, dtype=torch.bfloat16)
    w = 1 + normal(g, H, spread=0.2)
    y, _, rstd = layer.rms_norm(x, w)
    _, ref, v = norm_ref(x[rows], None, w, 1e-6)
    within(y[rows], v, v.abs() * (U[torch.bfloat16] + 80 * E) + TINY[torch.bfloat16], "y")
    assert int((rstd < 999).sum()) == 3
    grad, grad_w = layer.rms_norm_backward(x, x, w, rstd)
    r = rstd[rows].double()[:, None]
    n, u = x[rows].double() * r, x[rows].double() * w.double()
    m = (u * n).mean(-1, keepdim=True)
    want = r * (u - n * m)
    size = r * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True))
    within(grad[rows], want, U[torch.bfloat16] * want.abs() + 96 * E * size + TINY[torch.bfloat16], "grad_x")
    within(grad_w, (x[rows].double() * n).sum(0), 1200 * E * (x[rows].double() * n).abs().sum(0) + 1e-40, "grad_w")


def test_rotary_past_32_bits():
    T, heads, D = 2200000, 8, 128                             # 2.25e9 values
    g = gen(42)
    x = torch.zeros(T, heads, D, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, T // 2, T - 1], device="cuda")
    x[rows] = normal(g, 3, heads, D, dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda")
    f = layer.rotary_frequencies(D)
    got = layer.rotary(x, pos, f)
    check_rotary(got[rows], x[rows], pos[rows], f, False, 1.0, False)
    assert int((got != 0).flatten(1).any(-1).sum()) == 3
