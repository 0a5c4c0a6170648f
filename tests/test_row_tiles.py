"""The choice of a row tile of the grouped 8-bit products (csrc/row_tiles.h, which the kernel
includes), on the CPU: for groups of any size the one that the tiles' true numbers give."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_top_router_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("c++")

pytestmark = pytest.mark.skipif(CXX is None, reason="needs a host compiler")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <cstdint>
#include <initializer_list>
#include "row_tiles.h"

int main() {
  long wrong = 0, counted = 0;
  // groups of the same size: the choice is that of one group's true numbers
  for (int height : {160, 256})
    for (int quarters : {5, 8})
      for (int groups : {1, 2, 7, 128, 1024})
        for (int64_t rows = 1; rows <= INT_MAX; rows += 1 + rows / 50) {
          const int64_t small = (rows + 63) / 64, large = (rows + height - 1) / height;
          const int s = groups * moe::choice_tiles(int(rows), 64), l = groups * moe::choice_tiles(int(rows), height);
          // (products that leave 32 bits would be negative or small)
          const bool fits = int64_t(s) * 4 <= INT_MAX && int64_t(l) * quarters <= INT_MAX;
          wrong += !fits || moe::takes_small(s, l, quarters) != (small * 4 <= large * quarters);
          // counts that stop at 2^16, a group's small tiles and two groups' large ones, do not agree with it
          const int64_t s16 = small < 65536 ? small : 65536, l16 = large < 65536 ? large : 65536;
          counted += (s16 * 4 <= l16 * quarters) != (small * 4 <= large * quarters);
        }
  std::printf("%ld %ld\n", wrong, counted);
}
"""


def test_the_choice_is_that_of_the_true_numbers(tmp_path):
    src, exe = tmp_path / "choice.cpp", tmp_path / "choice"
    src.write_text(PROGRAM)
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    wrong, counted = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert wrong == 0
    assert counted > 0  # the sizes reach what a bound on the counts gets wrong


def test_the_kernel_takes_the_rule():
    with open(os.path.join(CSRC, "fp8_gemm.h")) as f:
        text = f.read()
    assert text.count("choice_tiles(c, ") == 2 and text.count("takes_small(uniform(few), uniform(tiles), ") == 1
    assert "1 << 16" not in text
