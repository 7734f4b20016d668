"""The cross entropy over a vocabulary on a GPU against its definition in 64 bits.

Tolerances: a logit is off by SUMS of the magnitudes of its terms (truncating
additions in the tensor cores, 16 products at a time), and lse by the most that
one of its row's is (its weights are probabilities); each exponential by 2^-21
(the hardware's, and its argument's last place), the sums by a chain of
groups / 32 + 40 additions and rescalings of 2^-21 each, the logarithm and the
last subtraction by 2^-22 of the result.  Where the inputs are small integers
every logit is exact and only the latter remain.
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


def case(T, I, V, dtype, whole=False, seed=0):
    """Inputs, and z with its bound; whole: small integers over a power of two, whose products and sums are exact."""
    g = gen(T + 7 * I + 13 * V + seed)
    if whole:
        x = torch.randint(-2, 3, (T, I), generator=g, device="cuda").to(dtype)
        w = torch.randint(-2, 3, (V, I), generator=g, device="cuda").to(dtype) * 2.0 ** -round(math.log2(I) / 2)
    else:
        x, w = normal(g, T, I, dtype=dtype), normal(g, V, I, dtype=dtype, spread=3 * I ** -0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    # ignored ones, and the vocabulary's ends
    for i, v in enumerate((V - 1, -100, 0, V, -1, V + 64, 1 << 40, -(1 << 40))):
        if i < T:
            target[i if T > 1 else 0] = v if T > 1 else V - 1
    z = x.double() @ w.double().t()
    off = torch.zeros_like(z) if whole else sums(I, x.double().abs() @ w.double().abs().t())
    return x, w, target, z, off


def reference(z, target):
    V = z.shape[1]
    lse = torch.logsumexp(z, -1)
    counts = (target >= 0) & (target < V)
    at = z.gather(1, torch.where(counts, target, 0)[:, None])[:, 0]
    return torch.where(counts, lse - at, torch.zeros_like(lse)), lse, counts


def check_forward(loss, lse, z, off, target, what=""):
    want_loss, want_lse, counts = reference(z, target)
    groups = math.ceil(z.shape[1] / 32)
    bound = 1.1 * off.amax(-1) + (groups / 32 + 40) * 2.0 ** -21 + 4 * E * want_lse.abs()
    within(lse, want_lse, bound, f"lse {what}")
    within(loss, want_loss, counts * (bound + 1.1 * off.amax(-1) + 4 * E * (want_lse.abs() + z.abs().amax(-1))), f"loss {what}")
    assert (loss[~counts] == 0).all()


SIZES = [(1, 64, 8), (1, 1, 1), (3, 100, 130), (17, 256, 1000), (129, 1279, 517), (300, 520, 20000), (40, 64, 40000),
         (2049, 328, 2600), (5, 4096, 33001), (257, 72, 127), (1000, 640, 129), (33, 24, 19456), (64, 16, 19455)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("T,I,V", SIZES)
def test_forward(T, I, V, whole, dtype):
    x, w, target, z, off = case(T, I, V, dtype, whole)
    check_forward(*layer.linear_cross_entropy(x, w, target), z, off, target)


# small vocabularies whose runs of K are tiles of their own (T V at most 2^19, V at most 8192, T at most 512,
# I above 1024, above 1984 in the gradients too), and the first sizes that are not so
RUNS = [(1, 1025, 8192), (64, 2048, 8192), (64, 1032, 8193), (65, 2000, 8065), (65, 2000, 8066), (512, 1985, 1024), (513, 1984, 1000),
        (16, 7168, 257), (3, 6296, 4584), (200, 2664, 1363), (2, 1090, 17), (31, 2048, 1), (128, 2047, 4096), (160, 4096, 3000),
        (300, 2056, 40)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("T,I,V", RUNS)
def test_runs_of_their_own(T, I, V, whole, dtype):
    x, w, target, z, off = case(T, I, V, dtype, whole)
    loss, lse = layer.linear_cross_entropy(x, w, target)
    check_forward(loss, lse, z, off, target)
    g = gen(V)
    gl, gs = normal(g, T), normal(g, T)
    got = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs)
    check_backward(got, x, w, target, z, off, lse, gl, gs, dtype)
    one = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs, want=(False, True))
    assert one[0] is None and torch.equal(one[1], got[1])
    check_backward(layer.linear_cross_entropy_backward(None, x, w, target, lse, grad_lse=gs), x, w, target, z, off, lse, None,
                   gs, dtype)


@pytest.mark.parametrize("I,V", [(1100, 8192), (2048, 1000), (7168, 300)])
def test_runs_of_their_own_have_the_same_bits(I, V):
    T = 700
    x, w, target, *_ = case(T, I, V, BF)
    whole = layer.linear_cross_entropy(x, w, target)
    for lo, hi in ((0, 1), (333, 334), (3, 40), (5, 69), (5, 70), (100, 229), (0, 512), (0, 513)):
        part = layer.linear_cross_entropy(x[lo:hi], w, target[lo:hi])
        assert all(torch.equal(a, b[lo:hi]) for a, b in zip(part, whole)), (lo, hi)


def test_runs_of_their_own_with_nan_and_infinities():
    x, w, target, z, off = case(70, 2100, 1500, BF)
    x[13, 7] = float("nan")
    x[69, 2099] = float("inf")
    x[1] = float("nan")                    # an ignored token: its loss is still 0
    loss, lse = layer.linear_cross_entropy(x, w, target)
    keep = [i for i in range(70) if i not in (1, 13, 69)]
    check_forward(loss[keep], lse[keep], z[keep], off[keep], target[keep])
    assert loss[1] == 0 and torch.isnan(lse[1]) and torch.isnan(loss[13]) and not torch.isfinite(loss[69])
    # tokens without a gradient have none, whatever their logits
    target[:] = -100
    gx, gw = layer.linear_cross_entropy_backward(torch.ones(70, device="cuda"), x.nan_to_num(0.0, 0.0), w, target, lse)
    assert (gx == 0).all() and (gw == 0).all()


@pytest.mark.parametrize("V", [100, 20001])
def test_spread_logits(V):
    """Logits hundreds apart, equal ones, and one far above the rest at each end."""
    I, T = 64, 6
    x, w = torch.zeros(T, I, dtype=BF, device="cuda"), torch.zeros(V, I, dtype=BF, device="cuda")
    w[:, 0] = torch.linspace(-512, 512, V, device="cuda").to(BF)
    w[0, 1], w[V - 1, 2], w[V // 2, 3] = 300, 300, -400
    x[0, 0], x[1, 1], x[2, 2], x[3, 3], x[4, 0] = 1, 1, 1, 1, -1       # (row 5: all logits 0)
    target = torch.tensor([0, 0, 0, V // 2, V - 1, 7], device="cuda")
    z = x.double() @ w.double().t()
    loss, lse = layer.linear_cross_entropy(x, w, target)
    check_forward(loss, lse, z, torch.zeros_like(z), target)
    assert loss[1].item() <= 2.0 ** -20 and abs(lse[5].item() - math.log(V)) <= 4e-5


@pytest.mark.parametrize("I,V", [(1024, 1500), (520, 30000), (1279, 300)])
def test_tokens_do_not_depend_on_the_batch(I, V):
    T = 700
    x, w, target, *_ = case(T, I, V, BF)
    whole = layer.linear_cross_entropy(x, w, target)
    assert all(torch.equal(a, b) for a, b in zip(layer.linear_cross_entropy(x, w, target), whole))
    for lo, hi in ((0, 1), (333, 334), (699, 700), (3, 40), (100, 229), (0, 512), (5, 21), (5, 22), (5, 37), (5, 38), (5, 69),
                   (5, 70), (5, 133), (5, 134)):
        part = layer.linear_cross_entropy(x[lo:hi], w, target[lo:hi])
        assert all(torch.equal(a, b[lo:hi]) for a, b in zip(part, whole)), (lo, hi)


@pytest.mark.parametrize("lead,extra", [(0, 8), (8, 8), (1, 0), (0, 1), (3, 5)])
def test_strides(lead, extra):
    x, w, target, *_ = case(37, 200, 333, BF)
    want = layer.linear_cross_entropy(x, w, target)
    xs, ws = strided(x, extra, lead), strided(w, extra, lead)
    assert all(torch.equal(a, b) for a, b in zip(layer.linear_cross_entropy(xs, ws, target), want))
    g = normal(gen(5), 37)
    grads = layer.linear_cross_entropy_backward(g, x, w, target, want[1])
    assert all(torch.equal(a, b) for a, b in zip(layer.linear_cross_entropy_backward(g, xs, ws, target, want[1]), grads))


def test_rows_with_nan_and_infinities():
    x, w, target, z, off = case(70, 100, 1500, BF)
    x[13, 7] = float("nan")
    x[69, 99] = float("inf")
    x[1] = float("nan")                    # an ignored token: its loss is still 0
    loss, lse = layer.linear_cross_entropy(x, w, target)
    keep = [i for i in range(70) if i not in (1, 13, 69)]
    check_forward(loss[keep], lse[keep], z[keep], off[keep], target[keep])
    assert loss[1] == 0 and torch.isnan(lse[1]) and torch.isnan(loss[13]) and not torch.isfinite(loss[69])
    # an entry of the vocabulary that is shut off
    w2 = torch.zeros_like(w)
    w2[:, 0] = 1
    w2[700, 0] = -float("inf")
    x2 = torch.zeros(2, 100, dtype=BF, device="cuda")
    x2[:, 0] = 1
    loss, lse = layer.linear_cross_entropy(x2, w2, torch.tensor([3, 700], device="cuda"))
    assert abs(lse[0].item() - 1 - math.log(1499)) <= 4e-5 and loss[1] == float("inf")


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------

def check_backward(got, x, w, target, z, off, lse, g, gs, dtype):
    T, I = x.shape
    V = w.shape[0]
    counts = (target >= 0) & (target < V)
    g64 = torch.zeros(T, dtype=torch.float64, device="cuda") if g is None else torch.where(counts, g.double(), 0.0)
    spread = g64 + (0 if gs is None else gs.double())
    lse = lse.double()[:, None]
    p = torch.exp(z - lse)
    d = p * spread[:, None]
    # the logit's own error, the subtraction's and the exponential's; then d's rounding (binary16: of d scaled so
    # that the largest gradient is at least 2^13, steps of 2^-24 of that)
    fine = d.abs() * (1.1 * off + 2.0 ** -21 * (1 + (z - lse).abs()) + 4 * E) + 2 * E * spread.abs()[:, None] * p
    rows = torch.nonzero(counts)[:, 0]
    d[rows, target[rows]] -= g64[rows]
    fine[rows, target[rows]] += 4 * E * g64[rows].abs()
    top = max(float(spread.abs().max()), float(g64.abs().max()))
    coarse = fine * (1 + U[dtype]) + U[dtype] * d.abs() + (2.0 ** -37 if dtype == HF else 2.0 ** -126) * top
    x64, w64 = x.double(), w.double()
    if got[0] is not None:
        want, size = d @ w64, d.abs() @ w64.abs()
        within(got[0], want, 1.1 * coarse @ w64.abs() + sums(min(V, 32768), size) + math.ceil(V / 4096) * E * size
               + U[dtype] * want.abs() + TINY[dtype], "grad_x")
    if got[1] is not None:
        want, size = d.t() @ x64, d.abs().t() @ x64.abs()
        within(got[1], want, 1.1 * coarse.t() @ x64.abs() + sums(T, size) + U[dtype] * want.abs() + TINY[dtype], "grad_w")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("T,I,V", SIZES)
def test_backward(T, I, V, whole, dtype):
    x, w, target, z, off = case(T, I, V, dtype, whole)
    loss, lse = layer.linear_cross_entropy(x, w, target)
    g = gen(V)
    gl, gs = normal(g, T), normal(g, T)
    got = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs)
    check_backward(got, x, w, target, z, off, lse, gl, gs, dtype)
    small = gl * 2.0 ** -20                              # a mean over many tokens
    check_backward(layer.linear_cross_entropy_backward(small, x, w, target, lse), x, w, target, z, off, lse, small, None, dtype)
    check_backward(layer.linear_cross_entropy_backward(None, x, w, target, lse, grad_lse=gs), x, w, target, z, off, lse, None,
                   gs, dtype)
    # each gradient alone has the same bits
    one = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs, want=(True, False))
    assert one[1] is None and torch.equal(one[0], got[0])
    one = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs, want=(False, True))
    assert one[0] is None and torch.equal(one[1], got[1])
    assert layer.linear_cross_entropy_backward(gl, x, w, target, lse, want=(False, False)) == (None, None)


def test_small_probabilities_in_binary16():
    """The mean over many tokens of flat distributions: each d is far below binary16's smallest value."""
    T, I, V = 300, 64, 5000
    x, w, target, z, off = case(T, I, V, HF, True)
    x[2:], w[:] = x[2:] * 0.125, w * 0.125
    z = x.double() @ w.double().t()
    loss, lse = layer.linear_cross_entropy(x, w, target)
    gl = torch.full((T,), 2.0 ** -7, device="cuda")      # times p = 1/5000: 1.6e-6, and half of the tokens 2^-20 of that
    gl[::2] *= 2.0 ** -20
    got = layer.linear_cross_entropy_backward(gl, x, w, target, lse)
    check_backward(got, x, w, target, z, off, lse, gl, None, HF)


@pytest.mark.parametrize("I", [128, 2048])
@pytest.mark.parametrize("dtype", BOTH)
def test_a_gradient_that_all_tokens_share_is_not_rounded(dtype, I):
    """A mean's: with g halfway between two values of the type, every target's gradient would be off by half a step."""
    T, V = 256, 4096
    g = gen(17)
    x, w = normal(g, T, I, dtype=dtype), normal(g, V, I, dtype=dtype, spread=0.125 * I ** -0.5)
    target = torch.randperm(V, generator=g, device="cuda")[:T]
    share = 2.0 ** -12 * (1 + U[dtype])
    gl = torch.full((T,), share, device="cuda")
    loss, lse = layer.linear_cross_entropy(x, w, target)
    gx, gw = layer.linear_cross_entropy_backward(gl, x, w, target, lse)
    p = torch.exp(x.double() @ w.double().t() - lse.double()[:, None])
    d = p.clone()
    d[torch.arange(T, device="cuda"), target] -= 1
    # p at a target is lost at most (under half a step of 1), the others have their own rounding, then the last one
    # (and 2^-16 for the logits, the exponentials, the scale and the sums)
    lost = float(p[torch.arange(T, device="cuda"), target].max())
    assert lost <= 2.0 ** -10
    for got, want, size, one in ((gx, d @ w.double(), p @ w.double().abs(), w[target].double().abs()),
                                 (gw[target], (d.t() @ x.double())[target], (p.t() @ x.double().abs())[target], x.double().abs())):
        bound = share * (U[dtype] * want.abs() + (1 + U[dtype]) * ((lost + 2.0 ** -16) * one + (U[dtype] + 2.0 ** -16) * size)) + TINY[dtype]
        within(got, share * want, bound, "gradient")


@pytest.mark.parametrize("I", [64, 2048])
@pytest.mark.parametrize("loss_power,lse_power", [(-90, 90), (-50, 50), (50, -50), (90, -90), (-100, -100), (-30, 0)])
def test_gradients_far_apart(loss_power, lse_power, I):
    T, V = 70, 300
    x, w, target, z, off = case(T, I, V, BF)
    loss, lse = layer.linear_cross_entropy(x, w, target)
    g = gen(29)
    gl, gs = (normal(g, T).abs().clamp(min=0.01) * 2.0 ** k for k in (loss_power, lse_power))
    check_backward(layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs), x, w, target, z, off, lse, gl, gs, BF)
    check_backward(layer.linear_cross_entropy_backward(gl, x, w, target, lse), x, w, target, z, off, lse, gl, None, BF)


def test_ignored_tokens_have_no_gradient():
    T, I, V = 200, 256, 3000
    x, w, target, z, off = case(T, I, V, BF)
    target[50:] = -100
    loss, lse = layer.linear_cross_entropy(x, w, target)
    gx, gw = layer.linear_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, target, lse)
    assert (gx[50:] == 0).all()
    # the others' are those of the others alone
    gx2, gw2 = layer.linear_cross_entropy_backward(torch.ones(50, device="cuda"), x[:50], w, target[:50], lse[:50])
    check_backward((gx[:50], gw), x[:50], w, target[:50], z[:50], off[:50], lse[:50], torch.ones(50, device="cuda"), None, BF)
    check_backward((gx2, gw2), x[:50], w, target[:50], z[:50], off[:50], lse[:50], torch.ones(50, device="cuda"), None, BF)
    # all of them ignored; a row whose logits are not finite among them leaves grad_x alone
    target[:] = -100
    gx, gw = layer.linear_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, target, lse)
    assert (gx == 0).all() and (gw == 0).all()
    bad = lse.clone()
    bad[7] = float("nan")
    gx, gw = layer.linear_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, target, bad)
    assert (gx == 0).all() and (gw == 0).all()
    # infinite and zero incoming gradients
    gx, gw = layer.linear_cross_entropy_backward(torch.zeros(T, device="cuda"), x, w, target, lse, grad_lse=torch.zeros(T, device="cuda"))
    assert (gx == 0).all() and (gw == 0).all()
    g = torch.ones(T, device="cuda")
    g[3] = float("inf")
    gx, _ = layer.linear_cross_entropy_backward(None, x, w, target, lse, grad_lse=g)
    assert not torch.isfinite(gx[3].float()).any() and torch.isfinite(gx[4:].float()).all()


@pytest.mark.parametrize("T,I,V", [(40, 328, 500), (700, 520, 40000), (300, 1023, 1001)])
def test_calls_in_a_row_and_in_a_graph(T, I, V):
    g = gen(T + I)
    ws = [normal(g, V, I, dtype=BF, spread=I ** -0.5) for _ in range(3)]
    first = normal(g, T, I, dtype=BF)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")

    def chain(wait):
        x, out = first, []
        for w in ws:
            loss, lse = layer.linear_cross_entropy(x, w, target)
            wait()
            got = layer.linear_cross_entropy_backward(loss, x, w, target, lse, grad_lse=lse)
            wait()
            out += [loss, lse, *got]
            x = got[0]
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


def test_other_stream():
    x, w, target, *_ = case(300, 511, 1700, BF)      # (odd rows: a larger workspace)
    want = layer.linear_cross_entropy(x, w, target)
    gl = normal(gen(1), 300)
    want += layer.linear_cross_entropy_backward(gl, x, w, target, want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer.linear_cross_entropy(x, w, target)
        got += layer.linear_cross_entropy_backward(gl, x, w, target, got[1])
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    got = layer.linear_cross_entropy(x, w, target, stream=side)
    got += layer.linear_cross_entropy_backward(gl, x, w, target, got[1], stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_no_tokens():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(8, 64, dtype=BF, device="cuda")
    target, none = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = layer.linear_cross_entropy(x, w, target)
    assert loss.shape == (0,) and lse.shape == (0,)
    gx, gw = layer.linear_cross_entropy_backward(none, x, w, target, lse)
    assert gx.shape == (0, 64) and gw.shape == (8, 64) and (gw == 0).all()


def test_refusals():
    x, w = torch.ones(4, 64, dtype=BF, device="cuda"), torch.ones(8, 64, dtype=BF, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    loss, lse = layer.linear_cross_entropy(x, w, t)
    back = layer.linear_cross_entropy_backward
    for bad in (lambda: layer.linear_cross_entropy(x.float(), w, t), lambda: layer.linear_cross_entropy(x, w.half(), t),
                lambda: layer.linear_cross_entropy(x, w, t.int()), lambda: layer.linear_cross_entropy(x, None, t),
                lambda: back(loss.double(), x, w, t, lse), lambda: back(loss, x, w, t, lse.bfloat16()),
                lambda: back(loss, x, w, t, None), lambda: back(loss, x, w, t, lse, grad_lse=lse.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: layer.linear_cross_entropy(x, w[:, :63], t), lambda: layer.linear_cross_entropy(x, w, t[:3]),
                lambda: layer.linear_cross_entropy(x, w, t.view(4, 1)), lambda: layer.linear_cross_entropy(x.cpu(), w, t),
                lambda: layer.linear_cross_entropy(x, w.cpu(), t), lambda: layer.linear_cross_entropy(x[:1].expand(4, 64), w, t),
                lambda: layer.linear_cross_entropy(x, w, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]),
                lambda: back(None, x, w, t, lse), lambda: back(loss[:3], x, w, t, lse), lambda: back(loss, x, w, t, lse[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(layer.LayerError):
        layer.linear_cross_entropy(x, w[:0], t)


def test_past_32_bits():
    """A vocabulary's weight and gradient past 2^31 values, and more than 2^31 logits."""
    I, T = 256, 300
    V = (1 << 31) // I + 4321
    g = gen(9)
    x = normal(g, T, I, dtype=BF)
    w = torch.zeros(V, I, dtype=BF, device="cuda")
    at = torch.tensor([0, 1, 255, V // 2, V - 2, V - 1], device="cuda")
    w[at] = normal(g, 6, I, dtype=BF, spread=0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[:60] = at.repeat(10)
    loss, lse = layer.linear_cross_entropy(x, w, target)
    z = x.double() @ w[at].double().t()
    most = torch.cat([z, torch.zeros(T, 1, device="cuda", dtype=torch.float64)], 1)
    want = torch.logsumexp(torch.cat([z, torch.full((T, 1), math.log(V - 6), device="cuda", dtype=torch.float64)], 1), -1)
    off = sums(I, (x.double().abs() @ w[at].double().abs().t()).amax(-1))
    chain = (V / 64 / 32 + 40) * 2.0 ** -21
    within(lse, want, off + chain + 4 * E * want.abs(), "lse")
    picked = (x.double() * w[target].double()).sum(-1)
    within(loss, want - picked, 2 * off + chain + 4 * E * (want.abs() + most.abs().amax(-1)), "loss")
    gl = torch.ones(T, device="cuda")
    _, gw = layer.linear_cross_entropy_backward(gl, x, w, target, lse, want=(False, True))
    p = torch.exp(z - lse.double()[:, None])
    d = p.clone()
    for j in range(6):
        d[:, j] -= (target == at[j]).double()
    x64 = x.double()
    err = U[BF] * 1.1 * d.abs() + p * (off[:, None] + 2.0 ** -20 * (2 + want.abs()[:, None]))
    ref = d.t() @ x64
    within(gw[at], ref, err.t() @ x64.abs() + sums(T, d.abs().t() @ x64.abs()) + U[BF] * ref.abs(), "grad_w")
    # an entry that is no target: the same flat probability times the sum of x
    others = [v for v in (5, V // 3, V - 5) if v not in set(target.tolist())]
    flat = torch.exp(-lse.double())
    ref = (flat @ x64)[None].expand(len(others), -1)
    bound = (1.1 * U[BF] * flat) @ x64.abs() + sums(T, flat @ x64.abs())
    within(gw[others], ref, bound[None] + U[BF] * ref.abs() + 2.0 ** -20 * 20 * (flat @ x64.abs())[None], "grad_w elsewhere")


def test_many_tokens_past_32_bits():
    """More than 2^31 gradients of logits in the workspace; few tokens have one."""
    T, I, V = 600000, 16, 4096
    g = gen(10)
    x, w = normal(g, T, I, dtype=BF), normal(g, V, I, dtype=BF)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    at = torch.tensor([0, 255, T // 2, T - 2, T - 1], device="cuda")
    loss, lse = layer.linear_cross_entropy(x, w, target)
    z = x[at].double() @ w.double().t()
    off = sums(I, x[at].double().abs() @ w.double().abs().t())
    check_forward(loss[at], lse[at], z, off, target[at])
    gl = torch.zeros(T, device="cuda")
    gl[at] = normal(g, 5)
    gx, gw = layer.linear_cross_entropy_backward(gl, x, w, target, lse)
    assert int((gx != 0).any(-1).sum()) == 5
    check_backward((gx[at], None), x[at], w, target[at], z, off, lse[at], gl[at], None, BF)
    # grad_w: the other tokens add zeros; a sum over T in the tensor cores loses nothing to them
    check_backward((None, gw), x[at], w, target[at], z, off, lse[at], gl[at], None, BF)


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


def test_gradient_against_differences():
    g = gen(22)
    x, w = normal(g, 4, 10, dtype=HF).requires_grad_(), normal(g, 7, 10, dtype=HF).requires_grad_()
    target = torch.tensor([3, -100, 6, 0], device="cuda")
    c, cs = normal(g, 4), normal(g, 4)
    loss, lse = autograd.linear_cross_entropy(x, w, target)
    torch.autograd.backward([loss, lse], [c, cs])

    def f(x64, w64):
        z = x64 @ w64.t()
        want, lse64, _ = reference(z, target.cpu())
        return (want * c.cpu().double() + lse64 * cs.cpu().double()).sum()

    want = differences(f, [t.detach().cpu().double() for t in (x, w)])
    for got, ref in zip((x.grad, w.grad), want):
        # d and the result are rounded to 11 bits each; at most 10 terms of at most 4
        assert (got.cpu().double() - ref).abs().max() <= 2.0 ** -7 * (1 + ref.abs().max())


def test_autograd():
    g = gen(24)
    x, w = normal(g, 2, 3, 64, dtype=BF).requires_grad_(), normal(g, 50, 64, dtype=BF).requires_grad_()
    target = torch.tensor([[1, 2, 49], [-100, 0, 7]], device="cuda")
    loss, lse = autograd.linear_cross_entropy(x, w, target)
    assert loss.shape == lse.shape == (2, 3)
    (loss.sum() / 5).backward()                    # (a broadcast incoming gradient)
    flat = x.detach().view(6, 64)
    want = layer.linear_cross_entropy_backward(torch.full((6,), 1.0, device="cuda") / 5, flat, w.detach(), target.view(-1),
                                               lse.detach().view(-1))
    assert torch.equal(x.grad.view(6, 64), want[0]) and torch.equal(w.grad, want[1])
    x.grad = w.grad = None
    loss, lse = autograd.linear_cross_entropy(x, w, target)
    lse.square().sum().backward()                  # lse alone
    want = layer.linear_cross_entropy_backward(None, flat, w.detach(), target.view(-1), lse.detach().view(-1),
                                               grad_lse=2 * lse.detach().view(-1))
    assert torch.equal(x.grad.view(6, 64), want[0]) and torch.equal(w.grad, want[1])
    with pytest.raises(ValueError):
        autograd.linear_cross_entropy(x, w, target[:1])
    loss = autograd.linear_cross_entropy(x, w, target)[0].sum()
    grad, = torch.autograd.grad(loss, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        (loss + grad.float().pow(2).sum()).backward()
