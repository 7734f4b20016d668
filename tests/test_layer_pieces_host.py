"""The pieces of a vocabulary and the parts of its sums: which sizes of _ends.py take which, from the plan alone."""

import subprocess

import _ends
from invariant_mhc_aggregate_gb300 import _build, layer

PROGRAM = """
#include <cstdio>
#include "mhc_linear_plan.h"
int main() {
    long long T, I, V;
    while (std::scanf("%lld %lld %lld", &T, &I, &V) == 3) {
        const long long piece = mhc::linear::entropy_piece(T, V), pieces = (V + piece - 1) / piece;
        const mhc::linear::Plan p = mhc::linear::sum_plan(I, T, ((piece < V ? piece : V) + 63) / 64);
        std::printf("%lld %lld %u %lld\\n", piece, pieces, p.splits, (V - (pieces - 1) * piece + 63) / 64);
    }
}
"""


def ask(tmp_path, cases):
    (tmp_path / "pieces.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "pieces")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, "-o", exe, str(tmp_path / "pieces.cpp")], check=True)
    text = "".join("%d %d %d\n" % c for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    return [tuple(int(v) for v in line.split()) for line in out if line]


def test_sizes_take_their_ways(tmp_path):
    cases = [*(c + (None,) for c in _ends.PIECES), _ends.SHORT]
    for (T, I, V, pieces, parts, last), got in zip(cases, ask(tmp_path, [c[:3] for c in cases])):
        assert got[1:3] == (pieces, parts), (T, I, V, got)
        assert last is None or (got[3] == last and last < parts)
    assert {c[4] == 1 for c in _ends.PIECES} == {True, False} and all(c[3] > 1 for c in _ends.PIECES)


def test_pieces_are_legal(tmp_path):
    cases = [(T, 64, V) for T in (1, 7, 64, 1000, 4096, 6899, 6900, 27594, 27595, 131072, 131073, 1 << 24)
             for V in (1, 63, 64, 4096, 4097, 19456, 19457, 131072, 1 << 22)]
    for (T, _, V), (piece, pieces, parts, last) in zip(cases, ask(tmp_path, cases)):
        assert piece % 64 == 0 and 1 <= last <= -(-piece // 64) and (pieces - 1) * piece < V <= pieces * piece
        # 256 MB of d with few tokens, a tile of 256 entries for each pair of CTAs or 1 GB with more, 4096 entries at least
        assert piece <= max(1 << 27, T * 256 * 76) // T + 64 and (T * piece <= (1 << 29) + 64 * T or piece <= 4096)


def test_grad_w_by_rows_has_its_tiles():
    for T, I, F in _ends.BY_ROWS:
        assert I % 16 == 0 and -(-2 * F // 256) * -(-I // 256) >= 76


TOKENS = """
#include <cstdio>
#include "mhc_linear_plan.h"
int main() {
    long long N, M, kb;
    while (std::scanf("%lld %lld %lld", &N, &M, &kb) == 3) {
        using namespace mhc::linear;
        const Plan t = token_plan(N, M, kb), p = plan_of(N, M, kb, true, false), s = sum_plan(N, M, kb, 128);
        std::printf("%d %u %u %d %d %u %u %u %u\\n", int(t.pair), t.width, t.splits, int(token_apart(t, kb)), int(p.pair), p.width, p.splits,
                    s.width, s.splits);
    }
}
"""


def test_sums_over_tokens(tmp_path):
    """No accumulator of a gated grad_w takes more than 256 blocks; up to there the plan is the product's."""
    (tmp_path / "tokens.cpp").write_text(TOKENS)
    exe = str(tmp_path / "tokens")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, "-o", exe, str(tmp_path / "tokens.cpp")], check=True)
    cases = [(N, M, kb) for N in (1, 16, 264, 600, 1000, 1279, 2048, 7168) for M in (2, 48, 320, 1040, 3000, 4200, 28672)
             for kb in (1, 63, 255, 256, 257, 512, 513, 1024, 2048, 2049, 16384, 65537)]
    text = "".join("%d %d %d\n" % c for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    ways = set()
    for (N, M, kb), line in zip(cases, out):
        pair, width, parts, apart, p_pair, p_width, p_parts, s_width, s_parts = (int(v) for v in line.split())
        assert (pair, width) == (p_pair, p_width)
        if kb <= 256:
            assert parts == p_parts and not apart
        run = -(-kb // (s_parts if apart else parts))
        assert run <= 256 and not (apart and pair)
        assert s_width in (128, 256)                 # (an operand's rows along its columns come in panels of 64, two a tile)
        ways.add((pair, apart, parts > 1))
    assert ways >= {(1, 0, False), (1, 0, True), (0, 0, True), (0, 1, True)}
    cases = [(I, 2 * F, -(-T // 64)) for T, I, F, _ in _ends.RUNS]
    out = subprocess.run([exe], input="".join("%d %d %d\n" % c for c in cases), capture_output=True, text=True, check=True).stdout.split("\n")
    got = [tuple(int(v) for v in line.split()) for line in out if line]
    assert ["apart" if g[3] else "pair" if g[0] and g[2] > 1 else "" for g in got] == [c[3] for c in _ends.RUNS]
    assert {g[7] for g, c in zip(got, _ends.RUNS) if c[3] == "apart"} == {128, 256}


def test_workspaces_are_what_the_header_says():
    """8 bytes for 16 to 64 logits, or a small vocabulary's sums; d whole up to 2^27 values, else a piece of it."""
    _build.build_layer()
    lib = layer.load()
    for T in (1, 64, 65, 512, 513, 4096, 100000):
        for V in (1, 100, 1024, 8192, 8193, 19456, 131072):
            for I in (64, 1024, 1088, 2048, 7168, 1 << 20):
                n = lib.mhc_linear_cross_entropy_workspace(T, I, V, I, I, 1)
                if V <= 8192 and T <= 512 and T * V <= 1 << 19 and I > 1024:
                    # T V / (T + V) is at most 512 / 1.5, and there are at most I / 1024 + 1 runs
                    assert n <= 1.4 * 2 * I * (T + V) + 16 and 4 * T * V * -(-I // 1024) <= n <= 4 * T * V * -(-I // 1024) + 16
                else:
                    assert n <= 8 * T * -(-V // 16) + 4 * T + 16 and (T <= 64 or n <= 8 * T * -(-V // 32) + 4 * T + 16)
                d = lib.mhc_linear_cross_entropy_bwd_workspace(T, I, V, I, I, 0, 1, 1)
                whole = 2 * T * (V + 63)
                assert d <= max(whole, 4 * T * V * -(-I // 1024) + whole if T * V <= 1 << 19 else 0) + 64
                assert T * V <= 1 << 27 or d < 2 * T * V
