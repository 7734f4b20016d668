"""The cross entropy's gradients over several pieces of the vocabulary, and the gated product's grad_w by rows, against 64
bits (tolerances as in test_entropy_gpu.py and test_gated_gpu.py; the ways that the sizes take are in _ends.py)."""

import pytest
import torch

import _ends
from invariant_mhc_aggregate_gb300 import _build, layer
from test_entropy_gpu import BF, BOTH, HF, TINY, U, case, check_backward, gen, normal, sums
from test_gated_gpu import act_ref
from test_gated_gpu import test_backward as check_gated_backward

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()
    yield
    assert layer.wait_timeouts() == 0


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,I,V", [c[:3] for c in _ends.PIECES])
def test_pieces(T, I, V, dtype):
    x, w, target, z, off = case(T, I, V, dtype)
    _, lse = layer.linear_cross_entropy(x, w, target)
    g = gen(V)
    gl, gs = normal(g, T), normal(g, T)
    got = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs)
    check_backward(got, x, w, target, z, off, lse, gl, gs, dtype)
    one = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs, want=(True, False))
    assert one[1] is None and torch.equal(one[0], got[0])
    one = layer.linear_cross_entropy_backward(gl, x, w, target, lse, grad_lse=gs, want=(False, True))
    assert one[0] is None and torch.equal(one[1], got[1])


@pytest.mark.parametrize("dtype", BOTH)
def test_a_last_piece_of_fewer_blocks_than_parts(dtype):
    T, I, V = _ends.SHORT[:3]
    g = gen(31)
    x, w = normal(g, T, I, dtype=dtype), normal(g, V, I, dtype=dtype)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    at, entries = torch.tensor([0, 1, 3500, T - 1], device="cuda"), torch.tensor([0, 19455, 19456, V - 2, V - 1], device="cuda")
    target[1], target[T - 1], target[5] = V - 1, V - 2, 19456
    _, lse = layer.linear_cross_entropy(x, w, target)
    gl = torch.where(torch.arange(T, device="cuda") % 3 == 0, -1.0, 1.0)
    gx, gw = layer.linear_cross_entropy_backward(gl, x, w, target, lse)
    z = x[at].double() @ w.double().t()
    off = sums(I, x[at].double().abs() @ w.double().abs().t())
    check_backward((gx[at], None), x[at], w, target[at], z, off, lse[at], gl[at], None, dtype)
    z = x.double() @ w[entries].double().t()
    off = sums(I, x.double().abs() @ w[entries].double().abs().t())
    d = torch.exp(z - lse.double()[:, None]) * gl.double()[:, None]
    fine = d.abs() * (1.1 * off + 2.0 ** -21 * (1 + (z - lse.double()[:, None]).abs()) + 8 * E)
    hit = target[:, None] == entries
    d -= gl.double()[:, None] * hit
    coarse = fine * (1 + U[dtype]) + 4 * E * hit + U[dtype] * d.abs() + (2.0 ** -37 if dtype == HF else 2.0 ** -126)
    want, size = d.t() @ x.double(), d.abs().t() @ x.double().abs()
    bad = (gw[entries].double() - want).abs() > 1.1 * coarse.t() @ x.double().abs() + sums(T, size) + U[dtype] * want.abs() + TINY[dtype]
    assert not bad.any()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,I,F", _ends.BY_ROWS)
def test_gated_grad_w_by_rows(T, I, F, act, dtype):
    check_gated_backward(T, I, F, act, dtype)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,I,F", [c[:3] for c in _ends.RUNS])
def test_gated_grad_w_of_runs_of_tokens(T, I, F, dtype):
    check_gated_backward(T, I, F, "silu", dtype)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("offset", [0, 16, 2])
def test_gated_grad_w_at_any_alignment(offset, dtype):
    """By rows on 32 bytes, with its values on the lanes elsewhere; nothing beside it is written."""
    T, I, F = 130, 1040, 2100
    g = gen(7)
    x, w = normal(g, T, I, dtype=dtype), normal(g, 2 * F, I, dtype=dtype, spread=F ** -0.5)
    z, gy = normal(g, T, 2 * F, dtype=dtype), normal(g, T, F, dtype=dtype)
    room = torch.full((2 * F * I + 256,), float("nan"), dtype=dtype, device="cuda")
    first = 128 + offset // 2
    out = room[first:first + 2 * F * I].view(2 * F, I)
    lib = layer.load()
    need = lib.mhc_gated_linear_bwd_workspace(T, I, F, I, I, 0, 1, 0, 1)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert room.data_ptr() % 256 == 0 and work.data_ptr() % 256 == 0
    assert lib.mhc_gated_linear_bwd(gy.data_ptr(), x.data_ptr(), w.data_ptr(), z.data_ptr(), 0, out.data_ptr(), 0, work.data_ptr(), need,
                                    T, I, F, I, I, 2, 0 if dtype == BF else 1, torch.cuda.current_stream().cuda_stream) == 0
    assert room[:first].isnan().all() and room[first + 2 * F * I:].isnan().all()
    gate, up, g64 = z[:, :F].double(), z[:, F:].double(), gy.double()
    a, s = act_ref(gate, "silu")
    u = torch.cat([g64 * up * s, g64 * a], 1)
    fine = torch.cat([(g64 * up).abs(), g64.abs()], 1) * 2.0 ** -18 * (1 + gate.abs().repeat(1, 2)) + 4 * E * u.abs()
    coarse = fine + 1.01 * U[dtype] * u.abs() + TINY[dtype]
    want, size = u.t() @ x.double(), u.abs().t() @ x.double().abs()
    off = (out.double() - want).abs()
    assert (off <= sums(T, size) + coarse.t() @ x.double().abs() + U[dtype] * want.abs() + TINY[dtype]).all()


def test_pairs_behind_blocks_that_still_run():
    """Thousands of calls without a pause: the logits' gradients' CTA pairs start on SMs where blocks of the launch before them
    are still running, so that the two CTAs of a pair start apart.  Every call ends, with the same bytes."""
    T, I, V = 513, 1279, 32003                # (rows off 16 bytes: that launch lays them out again)
    x, w, target, _, _ = case(T, I, V, HF)
    target[::3] = -100
    _, lse = layer.linear_cross_entropy(x, w, target)
    gl = torch.full((T,), 0.25, device="cuda")
    want = layer.linear_cross_entropy_backward(gl, x, w, target, lse)
    torch.cuda.synchronize()
    for _ in range(6):
        for _ in range(2000):
            got = layer.linear_cross_entropy_backward(gl, x, w, target, lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
