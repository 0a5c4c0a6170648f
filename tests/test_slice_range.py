"""The buffer loads of the 8-bit products' slices, walked on the CPU by the kernels' own
rule (csrc/slice_range.h), the slices past a reduction's end among them. A lane of a raw
buffer load is out of range where its offset is at or past num_records less the scalar
offset, unsigned: no lane that the rule lets through may lie outside its operand."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")

pytestmark = pytest.mark.skipif(CXX is None, reason="needs a host compiler")

WALK = r"""
#include <cstdio>
#include <initializer_list>
#include "slice_range.h"
using moe::SliceRange;
constexpr uint32_t kPast = 0x80000000u;

// a rule without the end's: the slice's own offset beside an empty range
static SliceRange unchecked(int kt, int end, uint32_t bytes) {
  return {kt < end ? bytes : 0u, uint32_t(kt)};
}

// Loads of `bytes` at lane offset v that are in range and outside the operand, over rows x per slices.
template <class Rule>
static long outside(Rule rule, int rows, int K, int from, int end, int ahead, int unit) {
  long bad = 0;
  const int runs = (K + 127) / 128, per = unit == 16 ? 128 : 4, width = unit == 16 ? K : runs * 4;
  const uint32_t size = uint32_t(rows) * uint32_t(width);
  for (int kt = from; kt < end + ahead; ++kt) {
    const SliceRange r = rule(kt, end, size);
    for (int row = 0; row < 8; ++row)
      for (int c = 0; c < per; c += unit) {
        const bool none = row >= rows || (unit == 16 && kt < end && kt * 128 + c >= K);
        const uint32_t v = none ? kPast : uint32_t(row) * uint32_t(width) + uint32_t(c);
        const uint32_t s = r.slice * uint32_t(per);
        if (v >= uint32_t(r.bytes - s)) continue;  // zeros
        if (uint64_t(v) + s + unit > size) ++bad;
      }
  }
  return bad;
}

int main() {
  long bad = 0, seen = 0, wrong = 0;
  for (int rows : {1, 2, 7, 8})
    for (int K : {16, 112, 128, 144, 256, 1040, 4096})
      for (int unit : {16, 4}) {
        const int runs = (K + 127) / 128;
        for (int from = 0; from < runs; from += 3)
          for (int end = from + 1; end <= runs; end += from ? runs : 1) {
            bad += outside(moe::slice_range, rows, K, from, end, 32, unit);
            seen += outside(unchecked, rows, K, from, end, 32, unit);
          }
        for (int kt = 0; kt < runs; ++kt) {  // slices that are there are not touched
          const SliceRange r = moe::slice_range(kt, runs, 99u);
          wrong += r.bytes != 99u || r.slice != uint32_t(kt);
        }
      }
  std::printf("%ld %ld %ld\n", bad, seen, wrong);
}
"""


def test_no_lane_leaves_its_operand(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-I",
                    os.path.join(ROOT, "combine_top_router_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    bad, seen, wrong = map(int, subprocess.run([str(exe)], check=True, capture_output=True,
                                               text=True).stdout.split())
    assert bad == 0 and wrong == 0
    assert seen > 0  # the walk sees an offset that passes an empty range


def test_the_products_take_every_slice_by_the_rule():
    """No transfer of the 8-bit products is given an offset that the rule did not make."""
    csrc = os.path.join(ROOT, "combine_top_router_amd", "csrc")
    calls = []
    for name in ("fp8_gemm.h", "fp8_gemm.hip"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for head in ("load16(", "load4("):
            at = text.find(head)
            while at >= 0:
                end = text.index(";", at)
                call = " ".join(text[at:end].split())
                if "asm" not in call and "i32x4 rsrc" not in call:
                    calls.append(call)
                at = text.find(head, end)
    assert len(calls) == 6
    for call in calls:
        assert "slice * " in call and "uint32_t(kt)" not in call, call
