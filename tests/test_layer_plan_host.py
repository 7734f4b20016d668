"""The matrix product's plan (kernel, tile width, parts of K): a function of
the sizes alone, since the parts fix the order of the sums."""

import os
import re
import subprocess

import pytest

from invariant_mhc_aggregate_gb300 import _build

PROGRAM = """
#include <cstdio>
#include "mhc_linear_plan.h"
int main() {
    long long N, M, kb;
    int q_mn, by_row;
    while (std::scanf("%lld %lld %lld %d %d", &N, &M, &kb, &q_mn, &by_row) == 5) {
        const mhc::linear::Plan p = mhc::linear::plan_of(N, M, kb, q_mn != 0, by_row != 0);
        std::printf("%d %u %u\\n", int(p.pair), p.width, p.splits);
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """Built by the host's compiler with no CUDA header in sight: there is no device to ask."""
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    exe = str(d / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, "-o", exe, str(d / "plan.cpp")], check=True)

    def ask(cases):
        text = "".join("%d %d %d %d %d\n" % c for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(int(v) for v in line.split()) for line in out if line]
    return ask


SIZES = [1, 8, 24, 127, 128, 129, 257, 1000, 1024, 4096, 4097, 7168, 11008, 14336, 50000]
ROWS = [1, 2, 15, 16, 17, 64, 100, 129, 255, 256, 257, 300, 512, 700, 1024, 1500, 4096, 20000, 16777217]
BLOCKS = [1, 2, 7, 23, 24, 31, 32, 56, 64, 112, 700]


def test_a_rows_parts_do_not_depend_on_the_rows(plan):
    for N in SIZES:
        for kb in BLOCKS:
            for q_mn in (0, 1):
                got = {p[2] for p in plan([(N, M, kb, q_mn, 1) for M in ROWS])}
                assert len(got) == 1, (N, kb, got)


def test_plans_are_legal(plan):
    cases = [(N, M, kb, q, r) for N in SIZES for M in ROWS for kb in BLOCKS for q, r in ((0, 1), (1, 1), (1, 0))]
    for (N, M, kb, q_mn, by_row), (pair, width, parts) in zip(cases, plan(cases)):
        assert parts in (1, 2, 4, 8) and (parts == 1 or kb // parts >= 8)
        if pair:
            assert 128 <= width <= 256 and width % (128 if q_mn else 32) == 0
            assert by_row or parts == 1
        else:
            assert 16 <= width <= 256 and width % (64 if q_mn else 16) == 0
            assert -(-M // width) <= 65535


def test_the_launch_asks_for_the_device_only_to_size_a_grid():
    code = re.sub(r"//.*", "", open(os.path.join(_build.CSRC, "mhc_launch_linear.cu")).read())
    assert re.findall(r".*num_sms\(\).*", code) == [
        "    const uint32_t tiles = a.p_tiles * a.q_tiles, pairs = uint32_t(num_sms()) / 2;"]
