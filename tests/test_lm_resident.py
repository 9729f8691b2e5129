"""CPU: the table of how many clusters a device holds (csrc/resident.h), compiled alone: one
device's answers are not another's, and a query that failed is asked again."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "stream_compaction_decoupled_gb300", "csrc")

SOURCE = r"""
#include <cstdio>
#include "resident.h"
static gbs::ResidentTable<4, 8> table;
static int asked = 0;
static int get(int device, unsigned size, int answer) {
  return table.get(device, size, [&](unsigned s) { ++asked; return s == size ? answer : -1; });
}
int main() {
  int a = get(0, 1, 304), b = get(1, 1, 264), c = get(0, 1, 7), d = get(1, 1, 7);
  std::printf("%d %d %d %d asked %d\n", a, b, c, d, asked);
  asked = 0;
  a = get(2, 5, -1), b = get(2, 5, 28), c = get(2, 5, 7);
  std::printf("%d %d %d asked %d\n", a, b, c, asked);
  asked = 0;
  a = get(3, 8, 0), b = get(3, 8, 9), c = get(3, 7, 9);
  std::printf("%d %d %d asked %d\n", a, b, c, asked);
}
"""


def test_answers_are_kept_for_each_device_and_failures_are_not(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    assert out[0] == "304 264 304 264 asked 2"  # each device its own, asked once
    assert out[1] == "0 28 28 asked 2"          # a failed query: none for now, asked again
    assert out[2] == "0 0 9 asked 2"            # none at all is an answer, of that size alone
