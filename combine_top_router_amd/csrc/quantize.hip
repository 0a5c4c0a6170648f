// Rows and weight matrices to 8 bits with scales (fp8.h has the formulas).
//
//   rows      a scale for each 128 of a row's columns: 16 lanes hold a run, eight
//             values each, and agree on its largest magnitude among themselves
//   weights   a scale for each block of 128 x 128, stored output-major: a workgroup
//             takes a block, 8 x 8 values to a thread, and turns them over in
//             registers and LDS where the matrix comes as [inner, cols]
//
// Bound: HBM, one read and one write of each value. Rows 8192 x 7168 bf16: 37 us, 4.8 TB/s;
// 32 matrices 7168 x 2048 bf16, turned over: 262 us, 5.4 TB/s (eight-byte stores of 16 lanes make
// whole lines; the transposition costs nothing beside the memory).
#include <algorithm>

#include "../../include/moe.h"
#include "fp8.h"

namespace moe {
namespace {

template <int T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* x, int64_t ldx, uint32_t total,
                                                            int H, int runs, void* q, float* scale) {
  const int l = threadIdx.x & 15;
  const uint32_t step = gridDim.x * 16u;
  constexpr int kBatch = 4;  // runs whose loads are in flight together
  for (uint64_t b0 = blockIdx.x * 16u + (threadIdx.x >> 4); b0 < total; b0 += uint64_t(step) * kBatch) {
    Raw<T> r[kBatch];
    int64_t row[kBatch];
    int col[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint64_t b = b0 + uint64_t(u) * step;
      row[u] = b < total ? uint32_t(b) / uint32_t(runs) : 0;
      col[u] = b < total ? int(uint32_t(b) - uint32_t(row[u]) * uint32_t(runs)) * kRun + l * 8 : H;
      if (col[u] < H) r[u] = load8<T>(x, row[u] * ldx + col[u]);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (col[u] < H) values8<T>(r[u], v);
      const float s = scale_of(max16(magnitude(v)));
      if (col[u] < H) {
        store_fp8x8(q, row[u] * H + col[u], to_fp8x8(v, 1.f / s));
        if (l == 0) scale[row[u] * runs + col[u] / kRun] = s;
      }
    }
  }
}

// One 128 x 128 block of matrix blockIdx.z. rows x cols: the matrix as it lies in
// memory; TURN: its columns become the rows of q.
template <int T, bool TURN>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const void* w, int rows, int cols,
                                                               uint8_t* q, float* scale) {
  __shared__ uint32_t red[4];
  // rows of 128 bytes and 8 more: the 8-byte writes of 16 lanes, eight rows apart, spread over the banks
  __shared__ __attribute__((aligned(16))) uint8_t tile[kRun * (kRun + 8)];
  const int64_t base = int64_t(blockIdx.z) * rows * cols;
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
  const int r0 = int(blockIdx.y) * kRun + tr * 8, c0 = int(blockIdx.x) * kRun + tc * 8;
  float v[8][8];
  {
    Raw<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + i < rows && c0 < cols) raw[i] = load8<T>(w, base + int64_t(r0 + i) * cols + c0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < rows && c0 < cols) {
        values8<T>(raw[i], v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      }
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
  m = max16(m);
  m = max(m, uint32_t(__shfl_xor(int(m), 16, kWave)));
  m = max(m, uint32_t(__shfl_xor(int(m), 32, kWave)));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  const float s = scale_of(m), inv = 1.f / s;
  const int rb = (rows + kRun - 1) / kRun, cb = (cols + kRun - 1) / kRun;
  if (threadIdx.x == 0)
    scale[int64_t(blockIdx.z) * rb * cb +
          (TURN ? int64_t(blockIdx.x) * rb + blockIdx.y : int64_t(blockIdx.y) * cb + blockIdx.x)] = s;
  if constexpr (!TURN) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + i < rows && c0 < cols)
        store_fp8x8(q, base + int64_t(r0 + i) * cols + c0, to_fp8x8(v[i], inv));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i][j];
      *reinterpret_cast<uint2*>(tile + (tc * 8 + j) * (kRun + 8) + tr * 8) = to_fp8x8(t, inv);
    }
    __syncthreads();
    // an output row is a column of w: `rows` values long (a multiple of 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = i * 16 + tr, k = tc * 8;
      const int on = int(blockIdx.x) * kRun + n, ok = int(blockIdx.y) * kRun + k;
      if (on < cols && ok < rows)
        store_fp8x8(q, base + int64_t(on) * rows + ok,
                    *reinterpret_cast<const uint2*>(tile + n * (kRun + 8) + k));
    }
  }
}

}  // namespace

hipError_t launch_quantize_fp8(int dtype, const void* x, int64_t rows, int H, int64_t ldx, void* q,
                               float* scale, hipStream_t s) {
  const int runs = (H + kRun - 1) / kRun;
  const uint32_t total = static_cast<uint32_t>(rows * runs);
  const int grid = static_cast<int>(std::min<int64_t>((int64_t(total) + 15) / 16, device_cu_count() * 16));
  auto go = [&](auto t) {
    quantize_rows_kernel<decltype(t)::value><<<grid, 256, 0, s>>>(x, ldx, total, H, runs, q, scale);
    return hipGetLastError();
  };
  if (dtype == MOE_ROWS_F32) return go(std::integral_constant<int, 2>{});
  if (dtype == MOE_ROWS_F16) return go(std::integral_constant<int, 1>{});
  return go(std::integral_constant<int, 0>{});
}

hipError_t launch_quantize_fp8_weights(int dtype, const void* w, int mats, int rows, int cols,
                                       bool turn, void* q, float* scale, hipStream_t s) {
  const dim3 grid((cols + kRun - 1) / kRun, (rows + kRun - 1) / kRun, mats);
  auto go = [&](auto t, auto turned) {
    quantize_weights_kernel<decltype(t)::value, decltype(turned)::value>
        <<<grid, 256, 0, s>>>(w, rows, cols, static_cast<uint8_t*>(q), scale);
    return hipGetLastError();
  };
  auto by = [&](auto t) {
    return turn ? go(t, std::true_type{}) : go(t, std::false_type{});
  };
  if (dtype == MOE_ROWS_F32) return by(std::integral_constant<int, 2>{});
  if (dtype == MOE_ROWS_F16) return by(std::integral_constant<int, 1>{});
  return by(std::integral_constant<int, 0>{});
}

}  // namespace moe
