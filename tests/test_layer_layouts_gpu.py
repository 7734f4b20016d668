"""Layouts of the layer operators' arguments that a user has at hand: the same
bytes as from dense ones, or a refusal that names them."""

import pytest
import torch

from invariant_mhc_aggregate_gb300 import _build, autograd, layer

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build_layer()
    _build.build_torch()
    yield
    assert layer.wait_timeouts() == 0


def normal(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,D,pad", [(13, 6, 64, 0), (1, 3, 64, 0), (40, 1, 96, 8), (1000, 8, 128, 0), (7, 5, 34, 1),
                                           (129, 3, 80, 4)])
def test_rotary_of_heads_outermost(T, heads, D, pad, interleaved):
    """[heads,T,D] seen as [T,heads,D]: the layout of keys and queries of an attention."""
    rows = normal(T + heads, heads, T, D + pad)
    x = rows[..., :D].transpose(0, 1)
    pos = torch.arange(T, device="cuda") * 37
    f = layer.rotary_frequencies(D // 2 // 2 * 2)
    want = layer.rotary(x.contiguous(), pos, f, interleaved=interleaved)
    for stream in (None, torch.cuda.current_stream()):
        got = layer.rotary(x, pos, f, interleaved=interleaved, stream=stream)
        assert got.is_contiguous() and torch.equal(got, want)
    xg = x.detach().requires_grad_()
    out = autograd.rotary(xg, pos, f, interleaved=interleaved)
    assert torch.equal(out, want)
    out.backward(want)
    assert torch.equal(xg.grad, layer.rotary(want, pos, f, interleaved=interleaved, inverse=True))


def test_rotary_refuses_overlapping_heads():
    x = normal(1, 4, 64)
    pos, f = torch.arange(4, device="cuda"), layer.rotary_frequencies(64)
    for bad in (x.view(4, 1, 64).expand(4, 2, 64), x[:1].view(1, 1, 64).expand(4, 1, 64),
                x.as_strided((2, 2, 64), (64, 32, 1)), x.as_strided((2, 2, 64), (32, 64, 1)),
                x.as_strided((2, 3, 64), (64, 64, 1))):
        with pytest.raises(ValueError, match="strides"):
            layer.rotary(bad, pos[:bad.shape[0]], f)
