"""The order of the layer operators' launches, read from the sources: a launch
may start while the one before it runs, and everything earlier is complete and
visible to it only after its own wait."""

import os
import re

from invariant_mhc_aggregate_gb300 import _build

SOURCES = {os.path.basename(p): re.sub(r"//.*", "", open(p).read()) for p in _build.LAYER_DEPS if p.startswith(_build.CSRC)}


def test_dependents_start_only_after_a_wait():
    """One place lets the next launch start, right after the wait for everything before."""
    code = "".join(SOURCES.values())
    assert code.count("griddepcontrol.launch_dependents") == 1
    assert re.search(r'void pdl_enter\(\) \{\s*asm volatile\("griddepcontrol\.wait;" ::: "memory"\);\s*'
                     r'asm volatile\("griddepcontrol\.launch_dependents;" :::\);\s*\}', code)


def test_every_kernel_waits_before_it_works():
    kernels = 0
    for name in ("mhc_norm.cuh", "mhc_linear.cuh", "mhc_rotary.cuh"):
        for body in SOURCES[name].split("__global__")[1:]:
            kernels += 1
            assert len(re.findall(r"\bpdl_enter\(\);", body)) == 1, (name, body[:200])
            # nothing of the call's memory is touched before
            before = body[body.index("{"):body.index("pdl_enter();")]
            assert not re.search(r"ld_stream|__ldg|tensor_copy|bulk_copy|load_words|load_weight|ring_copy|load_p|load_q", before)
    assert kernels == 10
