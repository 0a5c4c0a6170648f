// What the buffer loads of one slice of an operand are given, in a kernel that
// also issues the loads of slices past the reduction's end (they bring zeros and cost no branch).
// Host and device; includes nothing of HIP.
#pragma once

#include <cstdint>

#include "host_device.h"

namespace moe {

// A raw buffer load is in range where its lane's byte offset is below num_records less
// the scalar offset, a difference of unsigned numbers: a scalar offset past the range
// would turn it over and let every lane through. So a slice at or past `end` has an
// empty range and no scalar offset, and one before it a scalar offset inside a row.
struct SliceRange {
  uint32_t bytes;   // num_records
  uint32_t slice;   // times the bytes of a slice in a row: the scalar offset
};

MOE_HOST_DEVICE constexpr SliceRange slice_range(int kt, int end, uint32_t bytes) {
  return kt < end ? SliceRange{bytes, static_cast<uint32_t>(kt)} : SliceRange{0u, 0u};
}

}  // namespace moe
