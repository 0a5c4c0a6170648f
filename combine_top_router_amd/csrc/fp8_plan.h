// Tile and split of a dense 8-bit product, chosen on the host from its sizes. Includes nothing of HIP.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <iterator>

namespace moe {
namespace {

constexpr int kPlanRun = 128;  // terms that share a scale: what a reduction is split by

// A tile shape with what its workgroups take, in microseconds: a slice with the whole chip at
// work, as a share of that on a quiet chip, and a workgroup's beginning and end without its
// stores; how much longer stores take where rows do not go out in 16-byte pieces.
struct Tile8 {
  int bm, bn;
  double slice, quiet, fixed, odd;
};
constexpr Tile8 kFastTiles[] = {{256, 256, 1.61, 0.66, 7.5, 10.4}, {128, 256, 0.83, 0.81, 4.8, 8.0},
                                {256, 128, 0.91, 0.71, 5.0, 6.7}, {128, 128, 0.54, 0.84, 3.3, 6.0}};
constexpr Tile8 kExactTiles[] = {{160, 256, 1.79, 0.88, 6.3, 9.0}, {256, 128, 1.59, 0.87, 5.4, 9.3},
                                 {128, 128, 0.97, 0.97, 3.9, 7.0}, {64, 256, 0.96, 0.98, 3.7, 7.9}};
constexpr int kSplits8[] = {1, 2, 3, 4, 6, 8, 12, 16};

struct Plan8 {
  int tile, splits, per_split;
};

// Tile and split of one product, from its sizes alone: the least estimated time. Rounds of
// workgroups over the chip (slower the more of it works: clock and memory), at least the
// memory's time, for a split the second launch. The figures are fits to timings of these kernels,
// bf16 out, 65 to 32768 rows, 128 to 12288 terms and 64 to 16384 columns: 113000 of the 8-bit sums' tiles and splits on
// 8040 products, 88000 of the full-width ones' on 6527. On them the choice is 1.4 and 1.9 % slower than
// the best on average (a twentieth of them by more than 8 and 9 %). Examples, fast: 8192x4096x4096 takes 256x256
// (120 us; 128x256 135), 1024x7168x4096 128x128 (37 us; 256x256 76); full width: 8192x8192x8192 160x256
// (911 us; 192x256, not kept, 944; 128x128 1072), 1024x7168x4096 128x128 (63 us; 160x256 99).
Plan8 make_plan8(int64_t M, int64_t N, int64_t K, bool exact, double cus) {
  const int64_t runs = (K + kPlanRun - 1) / kPlanRun, nw = (N + 7) / 8 * 8;
  const double mem = (double(M) * K + double(N) * K + double(M) * N * 2.0) / 5.0e6;
  Plan8 best{0, 1, static_cast<int>(runs)};
  double best_t = 1e300;
  static_assert(std::size(kExactTiles) == std::size(kFastTiles), "one loop over either");
  for (int t = 0; t < int(std::size(kFastTiles)); ++t) {
    const Tile8& c = exact ? kExactTiles[t] : kFastTiles[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (const int want : kSplits8) {
      if (want > 1 && want * 2 > runs) break;
      const int64_t per = (runs + want - 1) / want, s = (runs + per - 1) / per;
      const double full = std::floor(double(tiles * s) / cus), rest = double(tiles * s) - full * cus;
      const double out = double(std::min<int64_t>(c.bm, M)) * double(std::min<int64_t>(c.bn, N)) *
                         (s > 1 ? 4.0 : N % 8 ? 2.0 * c.odd : 2.0) / 16.5e6;  // one workgroup's stores
      double time = full * (double(per) * c.slice + c.fixed + cus * out);
      if (rest > 0)
        time += double(per) * c.slice * (c.quiet + (1.0 - c.quiet) * rest / cus) + c.fixed + rest * out;
      time = std::max(time, mem);
      if (s > 1) time += 6.3 + double(s) * double(M) * double(nw) * 4.0 / 4.5e6;
      if (time < best_t) {
        best_t = time;
        best = {t, static_cast<int>(s), static_cast<int>(per)};
      }
    }
  }
  return best;
}

}  // namespace
}  // namespace moe
