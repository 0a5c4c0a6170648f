"""Tile and split of the dense 8-bit products, chosen on the host (csrc/fp8_plan.h): the sizes
of the GPU tests reach every tile, as they say they do."""
import os
import shutil
import subprocess

import pytest

import fp8_sizes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")

pytestmark = pytest.mark.skipif(CXX is None, reason="needs a host compiler")

PROGRAM = r"""
#include <cstdio>
#include "fp8_plan.h"

int main() {
  long long M, K, N;
  int fast;
  while (std::scanf("%d %lld %lld %lld", &fast, &M, &K, &N) == 4) {
    const moe::Plan8 p = moe::make_plan8(M, N, K, !fast, 256);
    const moe::Tile8& t = fast ? moe::kFastTiles[p.tile] : moe::kExactTiles[p.tile];
    std::printf("%d %d %d %d\n", t.bm, t.bn, p.splits, p.per_split);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "combine_top_router_amd", "csrc"),
                    str(at / "plan.cpp"), "-o", str(at / "plan")], check=True)

    def ask(sizes):
        text = "".join(f"{int(f)} {m} {k} {n}\n" for f, m, k, n in sizes)
        out = subprocess.run([str(at / "plan")], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


@pytest.mark.parametrize("name", ["WALKS", "ODD_WALKS", "SINGLE", "SPLIT"])
def test_sizes_reach_the_tiles(plan, name):
    cases = getattr(fp8_sizes, name)
    for case, (bm, bn, splits, per) in zip(cases, plan([(c[0], *c[3:]) for c in cases])):
        _, m, n, M, K, N = case
        assert (bm, bn) == (m, n), case
        tiles = -(-M // bm) * -(-N // bn)
        assert K % 128 and (splits > 1) == (name == "SPLIT") and (N % 8 != 0) == (name == "ODD_WALKS"), case
        assert (tiles > 256) == name.endswith("WALKS"), case
        if name == "WALKS":
            assert M % 16 == 1, case


def test_every_tile_is_among_them():
    for name in ("WALKS", "ODD_WALKS", "SINGLE"):
        assert len({c[:3] for c in getattr(fp8_sizes, name)}) == 8
    assert len({c[:3] for c in fp8_sizes.SPLIT}) == 6


def test_splits_cover_the_reduction(plan):
    sizes = [(f, m, k, n) for f in (0, 1) for m in (65, 300, 5000) for k in (16, 144, 2048, 8208, 1 << 20)
             for n in (1, 100, 4096)]
    for (_, _, k, _), (_, _, splits, per) in zip(sizes, plan(sizes)):
        runs = -(-k // 128)
        assert splits >= 1 and (splits - 1) * per < runs <= splits * per
