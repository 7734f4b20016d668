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


TOGETHER = r"__syncwarp\(\)|wait_warp\(|__all_sync\(|__any_sync\(|group_sync\(|gated_chunk<"
APART = (r"load_residual<|\bemit<|emit_any<|emit_sum<|give_back\(\)|if \(lane == 0\)|n_ok \?|if \(ok\)|if \(n_ok|if \(there|if \(sectors"
         r"|if \(halves|prefetch_l2\(|row_head<|elect\(\)|entropy_tile\(|entropy_lanes<")
WHOLE = (r"tmem_ld\(|tmem_st\(|tmem_wait_ld\(|tmem_wait_st\(|entropy_add<|emit_tile<|sum_tile<|sum_columns<|row_tile<|gated_tile<")


def body(code, at):
    """The block that opens at or after `at`, and where it ends."""
    start = code.index("{", at)
    depth = 0
    for i in range(start, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[start + 1:i], i + 1
    raise AssertionError("no end")


def unrolled(code):
    """Every loop's body twice, so that what ends one round stands before the next."""
    out, at = "", 0
    for m in re.finditer(r"\bfor \(", code):
        if m.start() < at:
            continue
        depth, i = 0, m.end() - 1
        while True:
            depth += {"(": 1, ")": -1}.get(code[i], 0)
            i += 1
            if depth == 0:
                break
        out += code[at:i]
        if code[i:].lstrip().startswith("{"):
            inside, at = body(code, i)
            out += 2 * unrolled(inside)
        else:
            at = code.index(";", i) + 1
            out += 2 * code[i:at]
    return out + code[at:]


def test_tensor_memory_is_read_and_written_by_whole_warps():
    """tcgen05's loads, stores and waits are .aligned: undefined where a warp's lanes have come apart.  Between what only some
    lanes do (loads and stores at ragged edges, signals of one lane) and such an instruction stands something that brings
    them together."""
    functions = places = 0
    for name in ("mhc_linear.cuh", "mhc_linear_ends.cuh", "mhc_few.cuh"):
        code = SOURCES[name]
        for m in re.finditer(r"__device__ __forceinline__ void (\w+)\(|__global__ void __launch_bounds__\([^{;]*?\)\s+(\w+)\(", code):
            text, _ = body(code, m.end())
            if not re.search(WHOLE, text):
                continue
            functions += 1
            together = True            # (a caller is held to it where it calls; a tile's end is the last of its round)
            for t in re.finditer(f"({WHOLE})|({TOGETHER})|({APART})", unrolled(text)):
                if t.group(1):
                    places += 1
                    assert together, (name, m.group(1) or m.group(2), t.group(0))
                else:
                    together = t.group(2) is not None
    assert functions == 9 and places > 40


def test_a_pair_gives_up_its_right_to_allocate_after_both_have():
    """One CTA's relinquish_alloc_permit.cta_group::2 goes for the pair: the peer's allocation has to be behind it, or it never
    ends (no limit bounds it).  Between the two stands a barrier of the cluster."""
    code = "".join(SOURCES.values())
    alloc, _ = body(code, code.index("void tmem_alloc("))
    assert "relinquish" not in alloc
    assert code.count("tmem_alloc<2>(") == 1 and code.count("tmem_relinquish<2>(") == 1 and code.count("tmem_relinquish<1>(") == 2
    text, _ = body(SOURCES["mhc_linear.cuh"], SOURCES["mhc_linear.cuh"].index("pair_kernel("))
    first, last = (text.index(t) for t in ("tmem_alloc<2>(", "if (warp == kCopyP) umma::tmem_relinquish<2>();"))
    assert first < text.index("umma::cluster_sync();", first) < last < text.index("pdl_enter();")


def test_a_pairs_tensor_memory_is_allocated_and_freed_while_both_ctas_run():
    """tcgen05.alloc and dealloc of cta_group::2 work on both SMs: the kernel's first barrier of the cluster stands before the
    one, and its last after the other."""
    code = SOURCES["mhc_linear.cuh"]
    text, _ = body(code, code.index("pair_kernel("))
    assert len(re.findall(r"tmem_free<2>\(|tmem_alloc<2>\(", "".join(SOURCES.values()))) == 2
    first = text.index("umma::cluster_sync();")
    assert first < text.index("tmem_alloc<2>(") < text.index("umma::cluster_sync();", first + 1) < text.index("pdl_enter();")
    assert re.search(r"umma::cluster_sync\(\);\s*umma::fence_after_sync\(\);\s*if \(warp == kCopyP\) umma::tmem_free<2>\(tmem, kTmemColumns\);"
                     r"\s*umma::cluster_sync\(\);\s*$", text)
    # whole warps at the barrier, and behind it
    assert re.search(r"void cluster_sync\(\) \{\s*__syncwarp\(\);[^}]*__syncwarp\(\);\s*\}", SOURCES["mhc_umma.cuh"])
