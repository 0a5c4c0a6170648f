// Products of 8-bit operands on the matrix cores: dense, and grouped by expert.
#include <algorithm>
#include <iterator>

#include "fp8_gemm.h"

namespace moe {
namespace {

// Few rows (16 RB at most): bound by reading w once. A workgroup takes 16 columns, its
// wavefronts every eighth run of the reduction, straight into registers; their sums meet in LDS.
template <int RB>
__global__ __launch_bounds__(kThreads8) void fp8_rows_kernel(Fp8Args g) {
  constexpr int D = RB == 1 ? 4 : RB == 2 ? 3 : 2;  // runs in flight
  constexpr int ROW = 20;                           // floats of an LDS row: 16 and a gap
  __shared__ __attribute__((aligned(16))) float part[kWaves8][16 * RB * ROW];
  const int tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const int r15 = lane & 15, grp = lane >> 4;
  const int K = g.K, N = g.N, KT = g.runs, M = int(g.M);
  const int n0 = int(blockIdx.x) * 16;
  const uint8_t* pw = g.w0 + int64_t(min(n0 + r15, N - 1)) * K + grp * 16;
  const float* ps = g.s0 + int64_t(n0 / kRun) * KT;
  const uint8_t* pa[RB];
  const float* psa[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t r = min(i * 16 + r15, M - 1);
    pa[i] = g.a + r * K + grp * 16;
    psa[i] = g.sa + r * KT;
  }
  struct Run {
    u32x4 w[2], a[RB][2];
    float s[RB], sw;
  } ring[D];
  // run kt; past the end, and the chunks of 16 past K, zeros
  auto fetch = [&](Run& x, int kt) __attribute__((always_inline)) {
    const int left = K - kt * kRun - grp * 16;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const bool in = z * 64 < left;
      x.w[z] = u32x4{0, 0, 0, 0};
      if (in) x.w[z] = *reinterpret_cast<const u32x4*>(pw + int64_t(kt) * kRun + z * 64);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        x.a[i][z] = u32x4{0, 0, 0, 0};
        if (in) x.a[i][z] = *reinterpret_cast<const u32x4*>(pa[i] + int64_t(kt) * kRun + z * 64);
      }
    }
    const int k = min(kt, KT - 1);
    x.sw = ps[k];
#pragma unroll
    for (int i = 0; i < RB; ++i) x.s[i] = psa[i][k];
  };
  f32x4 sum[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(ring[d], wid + kWaves8 * d);
  for (int kt = wid; kt < KT; kt += kWaves8 * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Run& x = ring[d];
      // (a run past the end is all zeros: its product is 0, whatever its scales)
      if (kt + kWaves8 * d < KT) {
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const f32x4 p = run_product_exact(join(x.w[0], x.w[1]), join(x.a[i][0], x.a[i][1]));
          const float s = x.s[i] * x.sw;
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[i][q] = __builtin_fmaf(p[q], s, sum[i][q]);
        }
      }
      fetch(x, kt + kWaves8 * (d + D));
    }
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
    *reinterpret_cast<f32x4*>(&part[wid][(i * 16 + r15) * ROW + grp * 4]) = sum[i];
  __syncthreads();
  const int r = tid >> 1, c = (tid & 1) * 8;
  if (r >= 16 * RB || r >= M || n0 + c >= N) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kWaves8; ++w) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(&part[w][r * ROW + c]);
    const f32x4 y = *reinterpret_cast<const f32x4*>(&part[w][r * ROW + c + 4]);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i], v[4 + i] += y[i];
  }
  const Block b(g.e, r, n0 + c);
  if (g.e.vec) {
    float bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = g.e.bias ? g.e.bias[n0 + c + i] : 0.f;
    finish8(g.e, b, 0, 0, v, bias, b.res ? load8x16(b.res) : u32x4{0, 0, 0, 0});
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float one[1] = {v[i]};
      if (n0 + c + i < N) finish_column(g.e, b, 0, 1, 1, i, one, g.e.bias ? g.e.bias[n0 + c + i] : 0.f);
    }
  }
}

// ---- host

constexpr int kFewRows = 64;
#ifndef GBM
#define GBM 160
#endif

struct Tile8 {
  int bm, bn;
  double slice, fixed;  // microseconds: a slice, a tile's beginning and end
};
constexpr Tile8 kTiles8[] = {{256, 256, 1.0, 5.0}, {128, 256, 0.6, 4.0}, {256, 128, 0.6, 4.0}, {128, 128, 0.4, 3.0}};
constexpr int kSplits8[] = {1, 2, 3, 4, 6, 8, 12, 16};

struct Plan8 {
  int tile, splits, per_split;
};

// exact: the fp32 output's products, which the smallest tile alone has
Plan8 plan8(int64_t M, int64_t N, int64_t K, bool exact) {
  const int64_t runs = (K + kRun - 1) / kRun, cus = device_cu_count();
  const int64_t nw = (N + 7) / 8 * 8;
  Plan8 best{0, 1, static_cast<int>(runs)};
  double best_t = 1e300;
  for (int t = exact ? 3 : 0; t < int(std::size(kTiles8)); ++t) {
    const Tile8& c = kTiles8[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (const int want : kSplits8) {
      if (want > 1 && want * 2 > runs) break;
      const int64_t per = (runs + want - 1) / want, s = (runs + per - 1) / per;
      const int64_t rounds = (tiles * s + cus - 1) / cus;
      double time = double(rounds) * (double(per) * c.slice + c.fixed);
      if (s > 1) time += 2.0 + double(s) * double(M) * double(nw) * 4.0 / 5.0e6;
      if (time < best_t) {
        best_t = time;
        best = {t, static_cast<int>(s), static_cast<int>(per)};
      }
    }
  }
  return best;
}

template <int KIND, int BM, int BN, int NS, bool EXACT = false>
hipError_t launch8(const Fp8Args& g, int64_t tiles, hipStream_t s) {
  const int grid = static_cast<int>(std::min<int64_t>(tiles, device_cu_count()));
  if (KIND == kDense && !g.e.vec && g.splits == 1)
    fp8_kernel<BM, BN, NS, KIND, KIND != kDense, EXACT><<<grid, kThreads8, 0, s>>>(g);
  else
    fp8_kernel<BM, BN, NS, KIND, true, EXACT><<<grid, kThreads8, 0, s>>>(g);
  return hipGetLastError();
}

Fp8Args operands(const void* x, const float* sx, const void* w, const float* sw, int K, int N) {
  Fp8Args g{};
  g.a = static_cast<const uint8_t*>(x), g.sa = sx;
  g.w0 = static_cast<const uint8_t*>(w), g.s0 = sw;
  g.K = K, g.N = N, g.runs = (K + kRun - 1) / kRun;
  g.splits = 1, g.per_split = g.runs;
  return g;
}

bool rows_wide(const void* p, int64_t ld, int bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * bytes % 16 == 0);
}

}  // namespace

size_t linear_fp8_workspace_bytes(const moe_linear_fp8_desc& d) {
  if (d.rows <= kFewRows) return 0;
  // (either output type's, so that the sizes alone decide)
  const int splits = std::max(plan8(d.rows, d.cols, d.inner, false).splits,
                              plan8(d.rows, d.cols, d.inner, true).splits);
  return splits > 1 ? size_t(splits) * d.rows * ((d.cols + 7) / 8 * 8) * 4 : 0;
}

bool linear_fp8_launchable(const moe_linear_fp8_desc& d) {
  // tile ids in 32 bits, with the smallest tile and the most splits; the second launch's threads
  return ((d.rows + 127) / 128) * ((d.cols + 127) / 128) < (int64_t(1) << 26) &&
         d.rows * ((d.cols + 7) / 8) < (int64_t(1) << 32) - 64;
}

hipError_t launch_linear_fp8(const moe_linear_fp8_desc& d, const void* x, const float* sx,
                             const void* w, const float* sw, const float* bias,
                             const void* residual, void* y, void* ws, hipStream_t s) {
  Fp8Args g = operands(x, sx, w, sw, d.inner, d.cols);
  g.M = d.rows;
  Epilogue& e = g.e;
  e.out = y, e.bias = bias, e.res = static_cast<const uint16_t*>(residual);
  e.ldo = d.ldy, e.ldr = d.ldr, e.act = d.act;
  e.f16 = d.dtype == MOE_ROWS_F16, e.out_f32 = d.y_f32 != 0;
  e.vec = d.cols % 8 == 0 && rows_wide(y, d.ldy, d.y_f32 ? 4 : 2) && rows_wide(residual, d.ldr, 2);
  if (d.rows <= kFewRows) {
    const int grid = (d.cols + 15) / 16;
    if (d.rows <= 16) fp8_rows_kernel<1><<<grid, kThreads8, 0, s>>>(g);
    else if (d.rows <= 32) fp8_rows_kernel<2><<<grid, kThreads8, 0, s>>>(g);
    else fp8_rows_kernel<4><<<grid, kThreads8, 0, s>>>(g);
    return hipGetLastError();
  }
  const Plan8 p = plan8(d.rows, d.cols, d.inner, d.y_f32 != 0);
  const Tile8& c = kTiles8[p.tile];
  g.tiles_m = static_cast<int>((d.rows + c.bm - 1) / c.bm);
  g.tiles_n = static_cast<int>((d.cols + c.bn - 1) / c.bn);
  g.splits = p.splits, g.per_split = p.per_split;
  g.part = static_cast<float*>(ws), g.nw = (d.cols + 7) / 8 * 8;
  const int64_t tiles = int64_t(g.tiles_m) * g.tiles_n * g.splits;
  hipError_t err;
  switch (p.tile) {
    case 0: err = launch8<kDense, 256, 256, 2>(g, tiles, s); break;
    case 1: err = launch8<kDense, 128, 256, 3>(g, tiles, s); break;
    case 2: err = launch8<kDense, 256, 128, 3>(g, tiles, s); break;
    default:
      err = e.out_f32 ? launch8<kDense, 128, 128, 4, true>(g, tiles, s)
                      : launch8<kDense, 128, 128, 4>(g, tiles, s);
      break;
  }
  if (err != hipSuccess || g.splits == 1) return err;
  const int64_t threads = d.rows * (g.nw / 8);
  fp8_join_kernel<<<static_cast<unsigned>((threads + 63) / 64), 64, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_gate_up_fp8(const moe_grouped_fp8_desc& d, const void* x, const float* sx,
                              const int32_t* src_row, const int32_t* offsets,
                              const int32_t* counts, const void* w1, const float* s1,
                              const void* w3, const float* s3, void* h, float* hs, hipStream_t s) {
  Fp8Args g = operands(x, sx, w1, s1, d.inner, d.cols);
  g.w1 = static_cast<const uint8_t*>(w3), g.s1 = s3;
  g.offsets = offsets, g.counts = counts, g.groups = d.num_groups;
  g.m_cap = d.m_cap, g.max_rows = static_cast<int>(std::min<int64_t>(d.max_rows, INT32_MAX));
  g.gather = src_row, g.top_k = d.top_k, g.tokens = d.num_tokens;
  g.h = static_cast<uint8_t*>(h), g.hs = hs;
  if (d.fast) return launch8<kGated, 256, 256, 2>(g, INT64_MAX, s);
  return launch8<kGated, GBM, 256, 2, true>(g, INT64_MAX, s);
}

hipError_t launch_down_fp8(const moe_grouped_fp8_desc& d, const void* h, const float* hs,
                           const int32_t* offsets, const int32_t* counts, const void* w2,
                           const float* s2, void* y, hipStream_t s) {
  Fp8Args g = operands(h, hs, w2, s2, d.inner, d.cols);
  g.offsets = offsets, g.counts = counts, g.groups = d.num_groups;
  g.m_cap = d.m_cap, g.max_rows = static_cast<int>(std::min<int64_t>(d.max_rows, INT32_MAX));
  g.e.out = y, g.e.ldo = d.cols, g.e.vec = true;
  return launch8<kGrouped, 256, 256, 2>(g, INT64_MAX, s);
}

}  // namespace moe
