"""CPU: how the selective scan splits rows into parts (csrc/lm.h), compiled alone: by the blocks that
run, and that an SM holds, at the number of states and the type that are asked for."""
import os
import random
import shutil
import subprocess

import pytest

from stream_compaction_decoupled_gb300 import _build

SOURCE = r"""
#include <cstdio>
#include "lm.h"
using namespace gbs;
int main() {
  long long B, T, D, N, G;
  while (std::scanf("%lld %lld %lld %lld %lld", &B, &T, &D, &N, &G) == 5) {
    for (int es : {2, 4}) {
      const SscForwardPlan f = ssc_forward_plan(B, T, D, N, G, es, false), s = ssc_forward_plan(B, T, D, N, G, es, true);
      const SscSplit b = ssc_backward_split(B, T, D, N, G, es);
      std::printf("%lld %lld %d %lld %lld %d %lld %lld %zu %zu\n", f.split.parts, f.split.tiles, f.lanes, s.split.parts, s.split.tiles,
                  s.lanes, b.parts, b.tiles, ssc_temp_bytes(B, T, D, N, G, es, false), ssc_temp_bytes(B, T, D, N, G, es, true));
    }
    std::printf("%zu %zu\n", ssc_temp_bytes(B, T, D, N, G, 0, false), ssc_temp_bytes(B, T, D, N, G, 0, true));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """ask(sizes): for each (B, T, D, N, G) a dict by bytes of a value, and the scratch of any type."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    d = tmp_path_factory.mktemp("parts")
    (d / "t.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", _build.CSRC, "-isystem", cuda, "-o", str(d / "t"), str(d / "t.cpp")],
                   check=True)

    def call(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        lines = subprocess.run([str(d / "t")], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        rows = [list(map(int, line.split())) for line in lines]
        return [({2: rows[k], 4: rows[k + 1]}, rows[k + 2]) for k in range(0, len(rows), 3)]
    return call


FORWARD = [  # what fills the device as it is, is one part; (sizes, bytes of a value, parts)
    ((12, 1024, 2048, 32, 1), 2, 1), ((8, 1024, 2048, 32, 1), 2, 1), ((8, 1024, 2048, 64, 1), 2, 1), ((8, 1024, 2048, 128, 1), 2, 1),
    ((4, 1024, 2048, 128, 1), 2, 1), ((8, 1024, 2048, 64, 1), 4, 1), ((4, 1024, 2048, 128, 1), 4, 1), ((8, 128, 2048, 16, 1), 2, 1),
    ((8, 2048, 2048, 16, 1), 2, 8)]
BACKWARD = [((8, 2048, 2048, 16, 1), 2, 1), ((4, 1024, 2048, 128, 1), 2, 1), ((4, 1024, 2048, 64, 1), 4, 1), ((7, 2048, 1024, 16, 1), 2, 8)]


def test_measured_sizes_get_the_parts_that_were_quickest(ask):
    for (_, es, parts), (by, _) in zip(FORWARD, ask([s for s, _, _ in FORWARD])):
        assert by[es][0] == parts
    for (_, es, parts), (by, _) in zip(BACKWARD, ask([s for s, _, _ in BACKWARD])):
        assert by[es][6] == parts


def test_parts_hold_all_tiles_and_the_scratch_all_parts(ask):
    r = random.Random(1)
    sizes = [(r.randint(1, 64), r.choice([0, 1, 15, 16, 17, 127, 128, 129, r.randint(1, 70000)]), 2 * r.randint(1, 3000),
              r.randint(1, 128), r.choice([1, 2])) for _ in range(400)] + [(1, 1 << 30, 8, 16, 1), (1 << 20, 3, 64, 16, 1)]
    for (b, t, d, n, g), (by, any_type) in zip(sizes, ask(sizes)):
        tiles = -(-t // 16)
        for es, row in by.items():
            for parts, each in (row[0:2], row[3:5], row[6:8]):
                assert parts >= 1 and parts * each >= tiles and (parts == 1 or ((parts - 1) * each < tiles and each >= 2))
            assert {row[2], row[5]} <= {2, 4} and (n <= 16 or row[2] == row[5] == 4)
            for parts in (row[0], row[3]) if es == 2 else (row[0],):
                assert row[8] >= 4 * b * (parts - 1) * (d * n + d + 1)
            assert any_type[0] >= row[8] and any_type[1] >= row[9]
            assert row[9] >= 4 * b * ((row[6] - 1) * (d * n + d + 1) + row[6] * d * (n + 2))
