"""What the layer operators' kernels do with whole warps, read from the
sources: the instructions that want all lanes of a warp find them together."""

import os
import re

from invariant_mhc_aggregate_gb300 import _build

SOURCES = {os.path.basename(p): re.sub(r"//.*", "", open(p).read()) for p in _build.LAYER_DEPS if p.startswith(_build.CSRC)}
TENSOR = ("mhc_linear.cuh", "mhc_linear_ends.cuh", "mhc_few.cuh", "mhc_gated.cuh", "mhc_entropy.cuh")


def test_a_warp_ends_a_wait_with_one_answer():
    """A lane's own limit may run out just when another lane gets through; a warp whose lanes go different ways then would
    wait for itself at the choice of a lane (elect.sync), without a limit."""
    assert re.search(r"bool wait_warp\(uint32_t bar, uint32_t parity\) \{\s*return __all_sync\(0xFFFFFFFFu, wait\(bar, parity\)\);\s*\}",
                     SOURCES["mhc_umma.cuh"])
    waits = 0
    for name in TENSOR:
        assert not re.search(r"umma::(try_)?wait\(", SOURCES[name]), name
        waits += SOURCES[name].count("umma::wait_warp(")
    assert waits == 13
