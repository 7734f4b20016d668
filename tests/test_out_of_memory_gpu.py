"""A call whose outputs or workspace do not fit raises torch's own error for that, on the current stream as on another.
(In a process of its own, whose memory is limited: other tests' memory is not in the way.)"""

import os
import subprocess
import sys

import pytest

from invariant_mhc_aggregate_gb300 import _build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import pytest, torch
from invariant_mhc_aggregate_gb300 import layer

x, w = (torch.ones(n, 64, device="cuda", dtype=torch.bfloat16) for n in (4096, 20000))
target = torch.zeros(4096, dtype=torch.int64, device="cuda")
lse = layer.linear_cross_entropy(x, w, target)[1]
g, side = torch.ones_like(lse), torch.cuda.Stream()
torch.cuda.synchronize()
torch.cuda.empty_cache()
# at most 64 MB more than is in use
torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / torch.cuda.mem_get_info()[1])
for stream in (None, side):
    for call in (lambda: layer.linear_cross_entropy_backward(g, x, w, target, lse, stream=stream),
                 lambda: layer.gated_linear_preact(x, w, stream=stream), lambda: layer.gated_linear(x, w, stream=stream),
                 lambda: layer.linear(x, w, stream=stream)):
        with pytest.raises(torch.cuda.OutOfMemoryError):
            call()
# and the next call goes through
assert layer.linear_cross_entropy(x[:8], w, target[:8])[0].shape == (8,)
assert layer.wait_timeouts() == 0
print("done")
"""


def test_torchs_error():
    _build.build_layer()
    _build.build_torch()
    out = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.endswith("done\n"), out.stderr[-2000:]
