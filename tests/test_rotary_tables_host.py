"""rotary_frequencies against its formulas, channel by channel, in 64 bits."""

import math

import pytest

from invariant_mhc_aggregate_gb300 import layer


@pytest.mark.parametrize("dim,factor,trained,fast,slow", [(64, 40.0, 4096, 32.0, 1.0), (128, 4.0, 32768, 32.0, 1.0),
                                                          (128, 8.0, 2048, 16.0, 2.0), (2, 4.0, 4096, 32.0, 1.0)])
def test_yarn_ramps_over_the_turns(dim, factor, trained, fast, slow):
    got = layer.rotary_frequencies(dim, scaling="yarn", factor=factor, trained=trained, fast=fast, slow=slow, device="cpu").double()
    between = 0
    for j in range(dim // 2):
        f = 10000.0 ** (-2 * j / dim)
        k = min(1.0, max(0.0, (trained * f / (2 * math.pi) - slow) / (fast - slow)))
        between += 0 < k < 1
        assert abs(float(got[j]) / (f * (k + (1 - k) / factor)) - 1) <= 2.0 ** -23
    assert between >= 8 or dim == 2


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk"])
def test_other_tables(scaling):
    dim, factor, base = 96, 8.0, 500000.0
    got = layer.rotary_frequencies(dim, base=base, scaling=scaling, factor=factor, device="cpu").double()
    if scaling == "ntk":
        base *= factor ** (dim / (dim - 2))
    for j in range(dim // 2):
        want = base ** (-2 * j / dim) / (factor if scaling == "linear" else 1.0)
        assert abs(float(got[j]) / want - 1) <= 2.0 ** -22
