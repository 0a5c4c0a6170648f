// Which row tile the grouped 8-bit products take: their large one or, where the groups
// are so small that it makes few more tiles, a small one with more stages (fp8_kernel has the
// figures). Host and device; includes nothing of HIP.
#pragma once

#include "host_device.h"

namespace moe {

// Tiles of `height` rows that a group counts for in the choice. Its rows are bounded, and not the
// counts, so that both tiles' counts keep their ratio; 1024 groups of tiles of
// 64 rows or more stay below 2^27.
MOE_HOST_DEVICE constexpr int choice_tiles(int rows, int height) {
  constexpr int kMost = 1 << 22;
  return ((rows < kMost ? rows : kMost) + height - 1) / height;
}

// The small tile, up to `quarters` / 4 times the large one's number.
MOE_HOST_DEVICE constexpr bool takes_small(int small_tiles, int large_tiles, int quarters) {
  return small_tiles * 4 <= large_tiles * quarters;
}

}  // namespace moe
