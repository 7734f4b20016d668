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


def test_groups_of_warps_meet_as_whole_warps():
    """The named barrier counts whole warps (bar.sync): after a store of some lanes they come together first."""
    assert re.search(r"void group_sync\(uint32_t id, uint32_t threads\) \{\s*__syncwarp\(\);\s*named_sync\(id, threads\);\s*\}",
                     SOURCES["mhc_umma.cuh"])
    meetings = 0
    for name in TENSOR:
        assert "named_sync(" not in SOURCES[name], name
        meetings += SOURCES[name].count("umma::group_sync(")
    assert meetings == 4
