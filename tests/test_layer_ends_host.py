"""The gated product's and the cross entropy's entry points on the host: what
they reject without touching a GPU, their workspaces, and the autograd
functions' own part with the kernels' calls replaced by torch formulas."""

import subprocess

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, autograd, layer

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 40          # a 256-byte aligned fake device address
GAP = 1 << 34        # keeps fake buffers apart


@pytest.fixture(scope="module")
def lib():
    _build.build_layer()
    return layer.load()


def test_compiled_marshalling_declines(lib):
    _build.build_torch()
    m = layer._compiled()
    x, s = torch.ones(2, 8, dtype=torch.bfloat16), torch.ones(2)
    t = torch.zeros(2, dtype=torch.int64)
    assert m.gated_linear(x, None, x, None, None, 0, -1, False) is None and m.gated_linear() is None
    assert m.gated_linear_backward(x, x, x, x, 0, True, True, True) is None
    assert m.linear_cross_entropy(x, x, t) is None and m.linear_cross_entropy(x, x, None) is None
    assert m.linear_cross_entropy_backward(s, x, x, t, s, None, True, True) is None
    with pytest.raises(ValueError, match="CUDA"):
        layer.gated_linear(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        layer.linear_cross_entropy(x, x, t)
    with pytest.raises(TypeError):
        layer.gated_linear(x.float(), x)
    with pytest.raises(ValueError, match="gate"):
        layer.gated_linear(x, x[:1])


def gated(lib, T=4, I=64, F=32, xs=None, ws=None, act=2, dtype=0, work=0, nbytes=0, **kw):
    a = dict(x=A, w=A + GAP, b=A + 2 * GAP, y=A + 3 * GAP, z=A + 4 * GAP)
    a.update(kw)
    xs, ws = (I if v is None else v for v in (xs, ws))
    return lib.mhc_gated_linear_fwd(a["x"], a["w"], a["b"], a["y"], a["z"], work, nbytes, T, I, F, xs, ws, act, dtype, 0)


def test_gated_refusals(lib):
    assert gated(lib, T=0, x=0, w=0, b=0, y=0, z=0) == OK
    for name in ("x", "w", "y"):
        assert gated(lib, **{name: 0}) == INVALID, name
    assert gated(lib, T=-1) == INVALID and gated(lib, I=0) == INVALID and gated(lib, F=0) == INVALID and gated(lib, F=-8) == INVALID
    assert gated(lib, act=4) == INVALID and gated(lib, act=-1) == INVALID and gated(lib, dtype=2) == INVALID
    assert gated(lib, xs=63) == INVALID and gated(lib, ws=63) == INVALID
    assert gated(lib, x=A + 1) == INVALID and gated(lib, b=A + 2 * GAP + 2) == INVALID and gated(lib, z=A + 4 * GAP + 1) == INVALID
    for other in (A, A + GAP, A + 2 * GAP, A + 4 * GAP):
        assert gated(lib, y=other + 16) == INVALID
    # w has 2 F rows and z 2 F columns: an output on their ends
    assert gated(lib, y=A + GAP + 63 * 64 * 2) == INVALID and gated(lib, y=A + 4 * GAP + 4 * 64 * 2 - 2) == INVALID
    assert gated(lib, F=(1 << 29) + 8) == UNSUPPORTED and gated(lib, I=(1 << 30) + 8) == UNSUPPORTED
    assert gated(lib, F=(1 << 62)) == UNSUPPORTED
    assert gated(lib, I=63) == INVALID
    need = lib.mhc_linear_workspace(4, 63, 64, 63, 63, 2, 1)
    assert need == (4 + 64) * 64 * 2
    assert gated(lib, I=63, work=A + 6 * GAP, nbytes=need - 1) == INVALID
    assert gated(lib, I=63, work=A + 6 * GAP + 8, nbytes=need) == INVALID
    assert gated(lib, I=63, work=A + 3 * GAP, nbytes=need) == INVALID


def test_gated_fp8_refusals(lib):
    p = [A + i * GAP for i in range(7)]                       # x sx w sw b y z

    def call(i=None, v=0):
        b = list(p)
        if i is not None:
            b[i] = v
        return lib.mhc_gated_linear_fp8_fwd(*b, 0, 0, 4, 64, 32, 64, 64, 2, 0, 0)

    for i in (0, 1, 2, 3, 5):
        assert call(i, 0) == INVALID, i
    assert call(1, p[1] + 2) == INVALID and call(5, p[3] + 255) == INVALID and call(5, p[3] + 252) == INVALID


def test_gated_backward_refusals(lib):
    T, I, F = 4, 64, 32
    need = lib.mhc_gated_linear_bwd_workspace(T, I, F, I, I, 1, 1, 1, 1)
    assert need == T * 64 * 2
    p = [A + i * GAP for i in range(8)]                       # g x w z gx gw gb ws

    def call(i=None, v=0, act=2, ws=need, T=T, xs=I, wst=I):
        b = list(p)
        if i is not None:
            b[i] = v
        return lib.mhc_gated_linear_bwd(*b, ws, T, I, F, xs, wst, act, 0, 0)

    for i in (0, 1, 2, 3, 7):
        assert call(i, 0) == INVALID, i
        assert call(i, 0, act=0) == INVALID, i                # (z without an activation too)
    assert call(ws=need - 2) == INVALID and call(act=5) == INVALID and call(T=-2) == INVALID
    assert call(xs=63) == INVALID and call(wst=0) == INVALID
    for out in (4, 5, 6, 7):
        for other in range(8):
            if other != out:
                assert call(out, p[other]) == INVALID, (out, other)
    ws = lib.mhc_gated_linear_bwd_workspace
    assert ws(700, 64, 36, 64, 64, 0, 0, 1, 1) == 11 * 72 * 4 + (16 - 11 * 72 * 4 % 16) % 16
    assert ws(700, 64, 36, 64, 64, 1, 0, 0, 1) == 700 * 80 * 2
    assert ws(700, 63, 36, 63, 63, 1, 1, 0, 1) == 700 * 80 * 2 + (700 + 72) * 64 * 2
    assert ws(0, 64, 36, 64, 64, 1, 1, 1, 1) == 0


def test_cross_entropy_refusals(lib):
    T, I, V = 4, 64, 1000
    need = lib.mhc_linear_cross_entropy_workspace(T, I, V, I, I, 1)
    assert need >= T * 4 + T * 8 * -(-V // 64)
    p = [A + i * GAP for i in range(6)]                       # x w target loss lse ws

    def call(i=None, v=0, ws=need, T=T, I=I, V=V, xs=64, wst=64, dtype=0):
        b = list(p)
        if i is not None:
            b[i] = v
        return lib.mhc_linear_cross_entropy_fwd(*b, ws, T, I, V, xs, wst, dtype, 0)

    for i in range(6):
        assert call(i, 0) == INVALID, i
    assert lib.mhc_linear_cross_entropy_fwd(*[0] * 6, 0, 0, I, V, 64, 64, 0, 0) == OK
    assert call(ws=need - 1) == INVALID and call(5, p[5] + 8) == INVALID and call(2, p[2] + 4) == INVALID
    assert call(T=-1) == INVALID and call(I=0) == INVALID and call(V=0) == INVALID and call(dtype=2) == INVALID
    assert call(xs=63) == INVALID and call(wst=63) == INVALID
    assert call(V=(1 << 30) + 1) == UNSUPPORTED and call(T=(1 << 30) + 1) == UNSUPPORTED
    for out in (3, 4, 5):
        for other in range(6):
            if other != out:
                assert call(out, p[other]) == INVALID, (out, other)
    ws = lib.mhc_linear_cross_entropy_workspace
    assert ws(4, 63, V, 63, 63, 1) == ws(4, 64, V, 64, 64, 1) + (4 + V) * 128
    assert ws(0, 64, V, 64, 64, 1) == 0


def test_cross_entropy_backward_refusals(lib):
    T, I, V = 4, 64, 40000
    need = lib.mhc_linear_cross_entropy_bwd_workspace(T, I, V, I, I, 1, 1, 1)
    assert need > 0 and lib.mhc_linear_cross_entropy_bwd_workspace(T, I, V, I, I, 0, 0, 1) == 0
    p = [A + i * GAP for i in range(9)]                       # gl gs x w target lse gx gw ws

    def call(v=None, ws=need, T=T, dtype=0, xs=64, wst=64):
        b = list(p)
        for i, a in (v or {}).items():
            b[i] = a
        return lib.mhc_linear_cross_entropy_bwd(*b, ws, T, I, V, xs, wst, dtype, 0)

    for i in (2, 3, 4, 5, 8):
        assert call({i: 0}) == INVALID, i
    assert call({0: 0, 1: 0}) == INVALID
    assert call({6: 0, 7: 0, 8: 0}, ws=0) == OK               # nothing to compute
    assert call(ws=need - 1) == INVALID and call({8: p[8] + 8}) == INVALID and call({0: p[0] + 2}) == INVALID
    assert call(T=-1) == INVALID and call(dtype=5) == INVALID and call(xs=0) == INVALID and call(wst=63) == INVALID
    for out in (6, 7, 8):
        for other in range(9):
            if other != out:
                assert call({out: p[other]}) == INVALID, (out, other)
    # the logits' gradients are in memory a piece of the vocabulary at a time
    ws = lib.mhc_linear_cross_entropy_bwd_workspace
    assert ws(4096, 4096, 1 << 20, 4096, 4096, 1, 1, 1) < 4096 * (1 << 20) // 2
    assert ws(0, 64, V, 64, 64, 1, 1, 1) == 0


# --- plans, which no device is asked for

PROGRAM = """
#include <cstdio>
#include "mhc_linear_plan.h"
int main() {
    long long N, M, kb;
    while (std::scanf("%lld %lld %lld", &N, &M, &kb) == 3) {
        const mhc::linear::Plan p = mhc::linear::sum_plan(N, M, kb);
        std::printf("%u %u %u %u\\n", p.width, p.splits, mhc::linear::few_lanes(N), mhc::linear::few_width(M));
    }
}
"""


def test_plans(tmp_path):
    (tmp_path / "plan.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, "-o", exe, str(tmp_path / "plan.cpp")], check=True)
    cases = [(N, M, kb) for N in (1, 16, 255, 1000, 4096, 9728, 9729, 16384, 19456, 19457, 28672, 65536, 151936, 1 << 24)
             for M in (1, 16, 17, 33, 64, 200, 4096, 70000) for kb in (1, 3, 64, 255, 256, 257, 516, 1500, 131072)]
    text = "".join("%d %d %d\n" % c for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for (N, M, kb), line in zip(cases, out):
        width, parts, lanes, few = (int(v) for v in line.split())
        assert width % 32 == 0 and 128 <= width <= 256
        assert 1 <= parts <= kb and -(-kb // parts) <= 256             # every part has a block, none more than 256
        assert lanes % 16 == 0 and 16 <= lanes <= 128
        # an SM's share of the weight is within one granule of 16 rows a round of the even one
        rounds = -(-N // (128 * 152))
        assert -(-(-(-N // lanes)) // 152) <= rounds and lanes * rounds <= -(-N // 152) + 16 * rounds + rounds
        assert few in (16, 32, 64) and (M > 64 or few >= M)


RUNS = """
#include <cstdio>
#include "mhc_linear_plan.h"
int main() {
    long long T, V, kb;
    while (std::scanf("%lld %lld %lld", &T, &V, &kb) == 3) {
        const long long runs = mhc::linear::entropy_runs(kb);
        std::printf("%d %lld %u %u\\n", int(mhc::linear::entropy_apart(T, V, kb)), runs, mhc::linear::apart_lanes(V, runs),
                    mhc::linear::apart_width(V, T, runs));
    }
}
"""


def test_runs_of_a_small_vocabulary(tmp_path):
    (tmp_path / "runs.cpp").write_text(RUNS)
    exe = str(tmp_path / "runs")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, "-o", exe, str(tmp_path / "runs.cpp")], check=True)
    cases = [(T, V, kb) for T in (1, 64, 65, 128, 512, 513, 1 << 20) for V in (1, 17, 1000, 4096, 8065, 8066, 8192, 8193, 1 << 24)
             for kb in (1, 16, 17, 32, 33, 112, 1 << 24)]
    text = "".join("%d %d %d\n" % c for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for (T, V, kb), line in zip(cases, out):
        apart, runs, lanes, width = (int(v) for v in line.split())
        assert runs == -(-kb // 16)
        assert apart == (kb > 16 and V <= 8192 and T <= 512 and T * V <= 1 << 19)
        assert lanes % 16 == 0 and 16 <= lanes <= 128 and width % 32 == 0 and 128 <= width <= 256


# --- autograd

B = torch.bfloat16


def gated_preact(x, w, bias=None, activation="silu", stream=None):
    z = x.float() @ w.float().t() + (0 if bias is None else bias)
    F = w.shape[0] // 2
    return (torch.relu(z[:, :F]) * z[:, F:]).to(x.dtype), z.to(x.dtype)


def gated_backward(g, x, w, z, activation="silu", bias=True, want=(True, True), stream=None):
    F = w.shape[0] // 2
    gate, up = z[:, :F].float(), z[:, F:].float()
    u = torch.cat([g.float() * up * (gate > 0), g.float() * torch.relu(gate)], 1)
    return ((u @ w.float()).to(x.dtype) if want[0] else None, (u.t() @ x.float()).to(x.dtype) if want[1] else None,
            u.sum(0) if bias else None)


@pytest.fixture
def formulas(monkeypatch):
    seen = []

    def entropy(x, w, target, stream=None):
        assert x.stride(1) == 1 and w.stride(1) == 1 and target.is_contiguous()
        z = x.float() @ w.float().t()
        lse = torch.logsumexp(z, -1)
        return torch.where(target >= 0, lse - z.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0), lse

    def entropy_backward(gl, x, w, target, lse, grad_lse=None, want=(True, True), stream=None):
        seen.append((gl, grad_lse, want))
        for t in (gl, grad_lse):
            assert t is None or t.is_contiguous()
        g = (torch.zeros_like(lse) if gl is None else gl) * (target >= 0)
        d = torch.exp(x.float() @ w.float().t() - lse[:, None]) * (g if grad_lse is None else g + grad_lse)[:, None]
        d[torch.arange(len(target)), target.clamp(min=0)] -= g
        return ((d @ w.float()).to(x.dtype) if want[0] else None, (d.t() @ x.float()).to(x.dtype) if want[1] else None)

    monkeypatch.setattr(layer, "gated_linear_preact", gated_preact)
    monkeypatch.setattr(layer, "gated_linear", lambda *a, **k: (seen.append("plain"), gated_preact(*a, **k)[0])[1])
    monkeypatch.setattr(layer, "gated_linear_backward", gated_backward)
    monkeypatch.setattr(layer, "linear_cross_entropy", entropy)
    monkeypatch.setattr(layer, "linear_cross_entropy_backward", entropy_backward)
    return seen


def rand(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(B)


def test_gated_autograd(formulas):
    x, w, b = rand(2, 3, 8).requires_grad_(), rand(10, 8).requires_grad_(), torch.rand(10).requires_grad_()
    y = autograd.gated_linear(x, w, bias=b, activation="relu")
    assert y.shape == (2, 3, 5) and formulas == []
    y.float().square().sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape and b.grad.shape == b.shape
    with torch.no_grad():                              # no gradient: z is not kept
        assert torch.equal(autograd.gated_linear(x, w, bias=b, activation="relu"), y)
    assert torch.equal(autograd.gated_linear(x.detach(), w.detach(), bias=b.detach(), activation="relu"), y)
    assert formulas == ["plain", "plain"]
    first = x.grad
    x.grad = None
    autograd.gated_linear(x, w.detach(), bias=b.detach()).float().square().sum().backward()
    assert torch.equal(x.grad, first)
    ctx = type("Saved", (), {"saved_tensors": (x, w, y), "needs_input_grad": (True,) * 5})()
    with pytest.raises(TypeError, match="gradient"):
        autograd.GatedLinear.backward(ctx, y.float())


def test_cross_entropy_autograd(formulas):
    x, w = rand(2, 3, 8).requires_grad_(), rand(9, 8).requires_grad_()
    target = torch.tensor([[0, 8, -100], [3, 4, 5]])
    loss, lse = autograd.linear_cross_entropy(x, w, target)
    assert loss.shape == lse.shape == (2, 3) and loss[0, 2] == 0
    (loss.sum() / 5).backward()
    assert formulas[-1][1] is None and formulas[-1][2] == (True, True)      # lse is not used: no zeros in its place
    want = torch.autograd.grad(torch.nn.functional.cross_entropy((x.float() @ w.float().t()).view(6, 9), target.view(6)), (x, w))
    for t, v in zip((x, w), want):
        assert (t.grad.float() - v.float()).abs().max() <= 2.0 ** -7 * v.float().abs().max()   # rounded to 8 bits on both sides
    loss, lse = autograd.linear_cross_entropy(x.detach(), w, target)
    lse.square().sum().backward()
    assert formulas[-1][0] is None and formulas[-1][2] == (False, True)
    loss, lse = autograd.linear_cross_entropy(x, w.detach(), target)
    loss.sum().backward()
    assert formulas[-1][2] == (True, False)
    with pytest.raises(ValueError):
        autograd.linear_cross_entropy(x, w, target.view(6))
    grad, = torch.autograd.grad(autograd.linear_cross_entropy(x, w, target)[0].sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        grad.float().square().sum().backward()
