"""The layer operators' library on the host: it builds, loads, exports what its
header declares, and rejects bad arguments without touching a GPU."""

import os
import re
import subprocess

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, layer

HEADER = os.path.join(_build.INCLUDE, "mhc_layer.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 40          # a 256-byte aligned fake device address
GAP = 1 << 34        # keeps fake buffers apart


@pytest.fixture(scope="module")
def lib():
    _build.build_layer()
    return layer.load()


def header_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return tuple(re.findall(r"^\s*MHC_API\s+\w+\s+(mhc_\w+)\s*\(", text, flags=re.M))


def test_exports(lib):
    assert header_functions() == layer.EXPORTS
    out = subprocess.run(["nm", "-D", "--defined-only", _build.LAYER_LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if line.strip()} == set(layer.EXPORTS)
    assert lib.mhc_layer_abi_version() == 1 and lib.mhc_layer_last_cuda_error() == 0


def test_compiled_marshalling_builds_and_declines(lib):
    _build.build_torch()
    m = layer._compiled()
    x, w = torch.ones(2, 8, dtype=torch.bfloat16), torch.ones(8)
    assert m.rms_norm(x, w, None, 1e-6, -1) is None          # not on a GPU: the checked path says so
    assert m.rms_norm(None, w, None, 1e-6, -1) is None
    assert m.linear(x, None, x, None, None, 0, None, -1, False) is None
    assert m.linear_backward(x, x, x, None, 0, True, True, True) is None
    assert m.rotary(x, w, w, False, 1.0, False) is None
    assert m.rms_norm() is None
    with pytest.raises(ValueError, match="CUDA"):
        layer.rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        layer.rotary(x.view(2, 1, 8), torch.zeros(2, dtype=torch.int64), torch.ones(4))
    with pytest.raises(TypeError):
        layer.linear(x.float(), x)


def test_kernels_are_built_without_fast_math_and_without_atomics():
    code = re.sub(r"//.*", "", "".join(open(p).read() for p in _build.LAYER_DEPS if p.startswith(_build.CSRC)))
    assert not re.findall(r"\batomic[A-Z]\w*\(", code) and not re.search(r"\bred\.", code)
    assert "tcgen05.mma" in code and "cp.async.bulk.tensor" in code and "mma.sync" not in code
    assert "use_fast_math" not in " ".join(_build.NVCC_FLAGS)


# --- RMS norm

def norm(lib, T=4, H=64, xs=None, rs=None, dtype=0, fp8=None, **kw):
    a = dict(x=A, r=A + GAP, w=A + 2 * GAP, y=A + 3 * GAP, s=A + 4 * GAP, t=A + 5 * GAP, d=A + 6 * GAP)
    a.update(kw)
    xs, rs = H if xs is None else xs, H if rs is None else rs
    if fp8 is None:
        return lib.mhc_rms_norm_fwd(a["x"], a["r"], a["w"], a["y"], a["t"], a["d"], T, H, xs, rs, 1e-6, dtype, 0)
    return lib.mhc_rms_norm_fp8_fwd(a["x"], a["r"], a["w"], a["y"], a["s"], a["t"], a["d"], T, H, xs, rs, 1e-6, fp8,
                                    dtype, 0)


@pytest.mark.parametrize("fp8", [None, 0, 128])
def test_norm_refusals(lib, fp8):
    assert norm(lib, T=0, fp8=fp8, x=0, r=0, w=0, y=0, s=0, t=0, d=0) == OK
    for name in ("x", "w", "y", "d"):
        assert norm(lib, fp8=fp8, **{name: 0}) == INVALID, name
    assert norm(lib, fp8=fp8, t=0) == INVALID                 # residual without total, and the other way round
    assert norm(lib, fp8=fp8, r=0) == INVALID
    assert norm(lib, fp8=fp8, x=A + 1) == INVALID
    assert norm(lib, fp8=fp8, w=A + 2 * GAP + 2) == INVALID
    assert norm(lib, fp8=fp8, T=-1) == INVALID
    assert norm(lib, fp8=fp8, H=0) == INVALID
    assert norm(lib, fp8=fp8, xs=63) == INVALID
    assert norm(lib, fp8=fp8, dtype=2) == INVALID
    assert norm(lib, fp8=fp8, H=32769) == UNSUPPORTED
    assert norm(lib, fp8=fp8, T=1 << 50, H=32768) == INVALID
    for out in ("y", "t", "d"):                               # an output on an input, or on another output
        assert norm(lib, fp8=fp8, **{out: A + 64}) == INVALID, out
        assert norm(lib, fp8=fp8, **{out: A + 2 * GAP}) == INVALID, out
    assert norm(lib, fp8=fp8, t=A + 3 * GAP + 32) == INVALID
    if fp8 is not None:
        assert norm(lib, fp8=fp8, s=0) == INVALID
        assert norm(lib, fp8=64) == UNSUPPORTED


def test_norm_backward_refusals(lib):
    T, H = 300, 64
    need = lib.mhc_rms_norm_bwd_workspace(T, H)
    assert need > 0 and need % (4 * H) == 0 and lib.mhc_rms_norm_bwd_workspace(1, H) == 0
    base = [A + i * GAP for i in range(8)]                    # g s w rstd gt gx gw ws

    def call(i=None, p=0, T=T, H=H, ws=need, gs=H, ss=H, dtype=0):
        b = list(base)
        if i is not None:
            b[i] = p
        return lib.mhc_rms_norm_bwd(*b, ws, T, H, gs, ss, dtype, 0)

    for i in (0, 1, 2, 3, 5, 6, 7):
        assert call(i, 0) == INVALID, i
    assert call(ws=need - 1) == INVALID
    assert call(7, base[7] + 4) == INVALID
    assert call(5, base[1]) == INVALID and call(6, base[2]) == INVALID and call(7, base[5]) == INVALID
    assert call(gs=63) == INVALID and call(ss=0) == INVALID and call(dtype=3) == INVALID
    assert call(H=40000, gs=40000, ss=40000) == UNSUPPORTED


# --- matrix product

def linear(lib, T=4, I=64, O=32, xs=None, ws=None, rs=None, act=0, dtype=0, work=0, nbytes=0, **kw):
    a = dict(x=A, w=A + GAP, b=A + 2 * GAP, r=A + 3 * GAP, y=A + 4 * GAP, z=A + 5 * GAP)
    a.update(kw)
    xs, ws, rs = (v if v is not None else d for v, d in ((xs, I), (ws, I), (rs, O)))
    return lib.mhc_linear_fwd(a["x"], a["w"], a["b"], a["r"], a["y"], a["z"], work, nbytes, T, I, O, xs, ws, rs, act,
                              dtype, 0)


def test_linear_refusals(lib):
    assert linear(lib, T=0, x=0, w=0, b=0, r=0, y=0, z=0) == OK
    for name in ("x", "w", "y"):
        assert linear(lib, **{name: 0}) == INVALID, name
    assert linear(lib, T=-1) == INVALID and linear(lib, I=0) == INVALID and linear(lib, O=0) == INVALID
    assert linear(lib, act=4) == INVALID and linear(lib, act=-1) == INVALID and linear(lib, dtype=2) == INVALID
    assert linear(lib, xs=63) == INVALID and linear(lib, ws=63) == INVALID and linear(lib, rs=31) == INVALID
    assert linear(lib, x=A + 1) == INVALID and linear(lib, b=A + 2 * GAP + 2) == INVALID
    for other in (A, A + GAP, A + 2 * GAP, A + 3 * GAP, A + 5 * GAP):
        assert linear(lib, y=other + 16) == INVALID
    assert linear(lib, I=(1 << 30) + 8) == UNSUPPORTED
    # operands whose rows do not start on 16 bytes need a workspace
    assert linear(lib, I=63) == INVALID
    assert linear(lib, x=A + 2) == INVALID
    need = lib.mhc_linear_workspace(4, 63, 32, 63, 63, 2, 1)
    assert need == (4 + 32) * 64 * 2
    assert linear(lib, I=63, work=A + 6 * GAP, nbytes=need - 1) == INVALID
    assert linear(lib, I=63, work=A + 6 * GAP + 8, nbytes=need) == INVALID
    assert linear(lib, I=63, work=A + 4 * GAP, nbytes=need) == INVALID       # on y


def test_linear_fp8_refusals(lib):
    p = [A + i * GAP for i in range(8)]                       # x sx w sw b r y z

    def call(i=None, v=0):
        b = list(p)
        if i is not None:
            b[i] = v
        return lib.mhc_linear_fp8_fwd(*b, 0, 0, 4, 64, 32, 64, 64, 32, 0, 0, 0)

    for i in (0, 1, 2, 3, 6):
        assert call(i, 0) == INVALID, i
    assert call(1, p[1] + 2) == INVALID and call(6, p[3]) == INVALID


def test_linear_workspace(lib):
    ws = lib.mhc_linear_workspace
    assert ws(7, 64, 32, 64, 64, 2, 1) == 0 and ws(7, 64, 32, 72, 80, 2, 1) == 0
    assert ws(7, 64, 32, 65, 64, 2, 1) == 7 * 64 * 2          # x alone
    assert ws(1, 63, 32, 63, 64, 2, 1) == 0                   # a single row has no stride
    assert ws(7, 64, 32, 64, 64, 2, 0) == (7 + 32) * 64 * 2   # pointers at any alignment
    assert ws(7, 64, 32, 64, 64, 1, 1) == 0 and ws(7, 72, 32, 72, 72, 1, 1) == (7 + 32) * 80
    bw = lib.mhc_linear_bwd_workspace
    assert bw(7, 64, 32, 0, 1, 1, 0, 1) == 0
    assert bw(7, 64, 32, 2, 1, 1, 0, 1) == 7 * 32 * 2         # u
    assert bw(7, 64, 32, 2, 0, 0, 1, 1) == 0                  # one run of rows: straight into grad_bias
    assert bw(700, 64, 32, 2, 0, 0, 1, 1) == 11 * 32 * 4
    assert bw(0, 64, 32, 2, 1, 1, 1, 1) == 0


def test_linear_backward_refusals(lib):
    T, I, O = 4, 64, 32
    need = lib.mhc_linear_bwd_workspace(T, I, O, 2, 1, 1, 1, 1)
    p = [A + i * GAP for i in range(8)]                       # g x w z gx gw gb ws

    def call(i=None, v=0, act=2, ws=need, T=T):
        b = list(p)
        if i is not None:
            b[i] = v
        return lib.mhc_linear_bwd(*b, ws, T, I, O, act, 0, 0)

    for i in (0, 1, 2, 3, 7):
        assert call(i, 0) == INVALID, i
    assert call(ws=need - 2) == INVALID and call(act=5) == INVALID and call(T=-2) == INVALID
    for out in (4, 5, 6, 7):
        for other in range(8):
            if other != out:
                assert call(out, p[other]) == INVALID, (out, other)


# --- rotary positions

def test_rotary_refusals(lib):
    def call(x=A, p=A + GAP, f=A + 2 * GAP, out=A + 3 * GAP, T=4, heads=2, D=64, R=64, xt=None, xh=None, ot=None, oh=None,
             dtype=0):
        xh, oh = (D if v is None else v for v in (xh, oh))
        xt, ot = (heads * D if v is None else v for v in (xt, ot))
        return lib.mhc_rotary(x, p, f, out, T, heads, D, R, xt, xh, ot, oh, 1.0, 0, 0, dtype, 0)

    assert call(T=0, x=0, p=0, f=0, out=0) == OK and call(heads=0) == OK
    for name in ("x", "p", "f", "out"):
        assert call(**{name: 0}) == INVALID, name
    assert call(R=63) == INVALID and call(R=66) == INVALID and call(R=-2) == INVALID
    assert call(D=70000, R=64) == UNSUPPORTED and call(heads=70000) == UNSUPPORTED
    assert call(T=-1) == INVALID and call(dtype=2) == INVALID
    assert call(xh=63) == INVALID and call(xt=127) == INVALID and call(oh=32) == INVALID and call(ot=64) == INVALID
    assert call(p=A + GAP + 4) == INVALID and call(x=A + 1) == INVALID
    assert call(out=A + 64) == INVALID                        # overlaps x without being x
    assert call(out=A, ot=256) == INVALID                     # x itself with other strides


def test_frequency_tables():
    f = layer.rotary_frequencies(8, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001]), rtol=1e-6)
    assert torch.equal(layer.rotary_frequencies(8, scaling="linear", factor=2.0, device="cpu"), f / 2)
    for bad in (lambda: layer.rotary_frequencies(7), lambda: layer.rotary_frequencies(0),
                lambda: layer.rotary_frequencies(8, scaling="cubic")):
        with pytest.raises(ValueError):
            bad()
