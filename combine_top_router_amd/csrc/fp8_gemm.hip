// Products of 8-bit operands on the matrix cores: dense, and grouped by expert.
//
//   z[m, n] = sum over runs b of sa[m, b] sw[n / 128, b] p_b[m, n],
//   p_b[m, n] = sum over k in [128 b, 128 b + 128) of a[m, k] w[n, k]
//
// A run is as long as one 16x16x128 instruction, or four of 16x16x32: its sum starts from zero, is scaled by
// an fp32 factor of its row and its block of columns and added in fp32, so that each product costs its matrix
// instructions and four vector additions for 16 x 16 outputs. Both operands lie with k last,
// w output-major; the product is taken as w a^T, which leaves four neighbouring columns of a row
// in a lane and 16-byte stores.
//
//   fp8_kernel       tiles of 64 .. 256 rows x 128 or 256 columns, one workgroup of eight
//                    wavefronts to a CU, that walks its tiles: two to four stages of a 128-long
//                    slice of both operands in LDS, filled by loads that go there directly, the
//                    chunks swizzled so that 16 rows' fragments lie in 16 bank groups; products in
//                    an order that frees fragments early (block_of); a tile's first slices are
//                    loaded during the epilogue of the tile before it.
//   fp8_rows_kernel  up to 64 rows: 16 or 32 columns to a workgroup, the reduction shared out among
//                    its wavefronts, each with a ring of its own.
//   fp8_join_kernel  the sums of a reduction split over workgroups, in order, and the epilogue.
//
// Two ways to a run's sum (run_product_exact, run_product): fp16 copies of the values, whose sums keep
// 24 bits; and where the caller asks for it (fast) the 8-bit instruction, at twice the rate, which loses 1.4e-5.
//
// Bound, with many rows: the matrix cores and their clock (1.7 to 2.1 GHz under this load), beside them the
// conversions to fp16. 8192x8192x8192 takes 917 us, 1200 TFLOP/s (a bf16 product of that size 1393);
// 65536x2048x7168 (few slices to a tile) 1660 us, and with a residual 1830: its loads come
// between the stores of a tile. fast: 452 us, 2430 TFLOP/s (a product with one scale for all, which
// needs no vector work, 2776), 910 and 1085 us; beside a product about five vector instructions are free
// there, the scaled addition and its scale take five: a sixth cost a fifth of the time.
// Few rows: one read of w. 16x7168x4096: 8.0 us, 3.7 TB/s; 32 experts' gate/up, 7168 -> 2048,
// 32 rows each: 167 us, 5.6 TB/s; down 103 us, 4.6 TB/s.
#include <algorithm>

#include "fp8_gemm.h"
#include "fp8_plan.h"

namespace moe {
namespace {

// Few rows (16 RB at most): bound by reading w once, and of a single call by the time that a
// chip full of first loads takes (16x7168x4096: 8.0 us, 29 MB). A workgroup takes 16 CB columns, its
// WAVES wavefronts an equal share of the runs each, through a ring of D runs in LDS that is
// the wavefront's own: no barrier until the wavefronts' sums meet in LDS at the end. (Fragments
// read from memory as they are needed, 16 rows x 64 bytes each, took half as long again:
// the transfers move whole lines, 8 rows x 128 bytes.)
template <int RB, int CB, int WAVES, int D>
__global__ __launch_bounds__(64 * WAVES) void fp8_rows_kernel(Fp8Args g) {
  constexpr int COLS = 16 * CB, ROW = COLS + 4;  // floats of a row of the sums: the columns and a gap
  constexpr int WB = CB * 16 * kRun, AB = RB * 16 * kRun, SLOT = WB + AB + 256;
  constexpr int NL = 2 * CB + 2 * RB + 1;  // wave-loads of a run
  constexpr int RING = D * SLOT, SUMS = 16 * RB * ROW * 4;
  static_assert(SUMS <= RING, "a wavefront's sums take its ring's place");
  __shared__ __attribute__((aligned(1024))) char smem[WAVES * RING];
  const int tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const int r15 = lane & 15, grp = lane >> 4;
  const int K = g.K, N = g.N, KT = g.runs, M = int(g.M);
  const int n0 = int(blockIdx.x) * COLS;
  const char* ring = smem + wid * RING;
  const uint32_t ring0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)) + wid * RING;
  // this lane's row in a wave-load of 8 rows x 128 bytes; the chunks are swizzled as the tiles' are
  const int lr = lane >> 3;
  const int nv = min(COLS, N - n0);
  const i32x4 rw = make_rsrc(g.w0 + int64_t(n0) * K, uint32_t(nv) * uint32_t(K));
  const i32x4 ra = make_rsrc(g.a, uint32_t(M) * uint32_t(K));
  const i32x4 rs = make_rsrc(g.sa, uint32_t(M) * uint32_t(KT) * 4u);
  uint32_t ow[2 * CB], oa[2 * RB];
#pragma unroll
  for (int i = 0; i < 2 * CB; ++i) {
    const int r = i * 8 + lr, c = (lane & 7) ^ ((r >> 1) & 7);
    ow[i] = r < nv ? uint32_t(r) * uint32_t(K) + uint32_t(c) * 16u : kPast;
  }
#pragma unroll
  for (int i = 0; i < 2 * RB; ++i) {
    const int r = i * 8 + lr, c = (lane & 7) ^ ((r >> 1) & 7);
    oa[i] = r < M ? uint32_t(r) * uint32_t(K) + uint32_t(c) * 16u : kPast;
  }
  const uint32_t os = lane < M && lane < 16 * RB ? uint32_t(lane) * uint32_t(KT) * 4u : kPast;
  // run kt into ring slot d; a run past the end, and a chunk past K, zeros
  auto fetch = [&](int d, int kt) __attribute__((always_inline)) {
    const int left = K - kt * kRun;
    const uint32_t at = ring0 + d * SLOT, slice = slice_range(kt, KT, 0).slice;
    auto upto = [&](i32x4 r) {
      r[2] = int(slice_range(kt, KT, uint32_t(r[2])).bytes);
      return r;
    };
#pragma unroll
    for (int i = 0; i < 2 * CB; ++i) {
      const int c = (lane & 7) ^ (((i * 8 + lr) >> 1) & 7);
      load16(upto(rw), c * 16 < left ? ow[i] : kPast, slice * kRun, at + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < 2 * RB; ++i) {
      const int c = (lane & 7) ^ (((i * 8 + lr) >> 1) & 7);
      load16(upto(ra), c * 16 < left ? oa[i] : kPast, slice * kRun, at + WB + i * 1024);
    }
    load4(upto(rs), os, slice * 4u, at + WB + AB);
  };
  f32x4 sum[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int c = 0; c < CB; ++c) sum[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* ps = g.s0 + int64_t(n0 / kRun) * KT;
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, wid + WAVES * d);
  const int f0 = r15 * kRun + ((grp ^ (r15 >> 1)) << 4);
  int d = 0;
  for (int kt = wid; kt < KT; kt += WAVES) {
    const float sw = ps[kt];
    wait_vmcnt<(D - 1) * NL>();
    const char* p = ring + d * SLOT;
    i32x8 w[CB];
#pragma unroll
    for (int c = 0; c < CB; ++c)
      w[c] = join(*reinterpret_cast<const u32x4*>(p + c * (16 * kRun) + f0),
                  *reinterpret_cast<const u32x4*>(p + c * (16 * kRun) + (f0 ^ 64)));
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const char* q = p + WB + i * (16 * kRun);
      const i32x8 a = join(*reinterpret_cast<const u32x4*>(q + f0), *reinterpret_cast<const u32x4*>(q + (f0 ^ 64)));
      const float s = *reinterpret_cast<const float*>(p + WB + AB + (i * 16 + r15) * 4) * sw;
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const f32x4 x = run_product_exact(w[c], a);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) sum[i][c][q4] = __builtin_fmaf(x[q4], s, sum[i][c][q4]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read
    fetch(d, kt + WAVES * D);
    d = d + 1 == D ? 0 : d + 1;
  }
  wait_vmcnt<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int c = 0; c < CB; ++c)
      *reinterpret_cast<f32x4*>(part + wid * (SUMS / 4) + (i * 16 + r15) * ROW + c * 16 + grp * 4) = sum[i][c];
  __syncthreads();
  for (int at = tid; at < 16 * RB * 2 * CB; at += 64 * WAVES) {
    const int r = at / (2 * CB), c = at % (2 * CB) * 8;
    if (r >= M || n0 + c >= N) continue;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(part + w * (SUMS / 4) + r * ROW + c);
      const f32x4 y = *reinterpret_cast<const f32x4*>(part + w * (SUMS / 4) + r * ROW + c + 4);
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
        if (n0 + c + i < N)
          finish_column(g.e, b, 0, 1, 1, i, one, g.e.bias ? g.e.bias[n0 + c + i] : 0.f);
      }
    }
  }
}

// ---- host

constexpr int kFewRows = 64;
// Row tile of the grouped products at full width. Their fp16 fragments leave no registers for more than
// 192 rows. Gate/up of 32 groups of 7168 -> 2048, with 128, 160, 192 rows a tile: groups of 160 rows 363, 282, 300 us; of
// 192 366, 379, 332; of 256 451, 455, 467; of 320 611, 544, 550; around 256 +- 16 520, 479, 484;
// of 512 859, 872, 856; of 2048 3238, 3130, 3122.
constexpr int kExactRows = 160;
constexpr int kFewTile = 64;  // row tile of the grouped products where groups are small

// The last few plans of this thread: a call asks for its plan several times over.
Plan8 plan8(int64_t M, int64_t N, int64_t K, bool exact) {
  struct Known {
    int64_t M, N, K, cus;
    bool exact;
    Plan8 p;
  };
  constexpr int kKnown = 16;
  thread_local Known known[kKnown] = {};
  thread_local int next = 0;
  const int64_t cus = device_cu_count();
  for (const Known& k : known)
    if (k.cus == cus && k.M == M && k.N == N && k.K == K && k.exact == exact) return k.p;
  const Plan8 p = make_plan8(M, N, K, exact, double(cus));
  known[next] = {M, N, K, cus, exact, p};
  next = (next + 1) % kKnown;
  return p;
}

template <int KIND, int BM, int BN, int NS, bool EXACT = false>
hipError_t launch8(const Fp8Args& g, int64_t tiles, hipStream_t s) {
  const int grid = static_cast<int>(std::min<int64_t>(tiles, device_cu_count()));
  if constexpr (KIND != kDense) {
    fp8_kernel<BM, BN, NS, KIND, true, EXACT, kFewTile><<<grid, kThreads8, 0, s>>>(g);
  } else if (!g.e.vec && g.splits == 1) {
    fp8_kernel<BM, BN, NS, KIND, false, EXACT, 0><<<grid, kThreads8, 0, s>>>(g);
  } else {
    fp8_kernel<BM, BN, NS, KIND, true, EXACT, 0><<<grid, kThreads8, 0, s>>>(g);
  }
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
  // (either kind of sums', so that the sizes alone decide)
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
  e.ldo = d.ldy, e.ldr = d.ldr, e.act = d.act & ~MOE_FP8_FAST;
  e.f16 = d.dtype == MOE_ROWS_F16, e.out_f32 = d.y_f32 != 0;
  e.vec = d.cols % 8 == 0 && rows_wide(y, d.ldy, d.y_f32 ? 4 : 2) && rows_wide(residual, d.ldr, 2);
  if (d.rows <= kFewRows) {
    // 32 columns to a workgroup halve what is read of x, where that leaves enough of them
    // (with the host's side, 16x7168x7168: 15.1 us, with 16 columns 17.6; 16x7168x4096: 12.3 and 10.3)
    auto go = [&](auto rb, auto depth) {
      constexpr int RB = decltype(rb)::value, D = decltype(depth)::value, W = kWaves8;
      if (d.cols >= 24 * device_cu_count())
        fp8_rows_kernel<RB, 2, W, D><<<(d.cols + 31) / 32, 64 * W, 0, s>>>(g);
      else
        fp8_rows_kernel<RB, 1, W, D><<<(d.cols + 15) / 16, 64 * W, 0, s>>>(g);
    };
    using std::integral_constant;
    if (d.rows <= 16) go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
    else if (d.rows <= 32) go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    else go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    return hipGetLastError();
  }
  const bool exact = !(d.act & MOE_FP8_FAST);
  const Plan8 p = plan8(d.rows, d.cols, d.inner, exact);
  const Tile8& c = exact ? kExactTiles[p.tile] : kFastTiles[p.tile];
  g.tiles_m = static_cast<int>((d.rows + c.bm - 1) / c.bm);
  g.tiles_n = static_cast<int>((d.cols + c.bn - 1) / c.bn);
  g.splits = p.splits, g.per_split = p.per_split;
  g.part = static_cast<float*>(ws), g.nw = (d.cols + 7) / 8 * 8;
  const int64_t tiles = int64_t(g.tiles_m) * g.tiles_n * g.splits;
  hipError_t err;
  if (exact) {
    switch (p.tile) {
      case 0: err = launch8<kDense, 160, 256, 2, true>(g, tiles, s); break;
      case 1: err = launch8<kDense, 256, 128, 3, true>(g, tiles, s); break;
      case 2: err = launch8<kDense, 128, 128, 4, true>(g, tiles, s); break;
      default: err = launch8<kDense, 64, 256, 3, true>(g, tiles, s); break;
    }
  } else {
    switch (p.tile) {
      case 0: err = launch8<kDense, 256, 256, 2>(g, tiles, s); break;
      case 1: err = launch8<kDense, 128, 256, 3>(g, tiles, s); break;
      case 2: err = launch8<kDense, 256, 128, 3>(g, tiles, s); break;
      default: err = launch8<kDense, 128, 128, 4>(g, tiles, s); break;
    }
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
  return launch8<kGated, kExactRows, 256, 2, true>(g, INT64_MAX, s);
}

hipError_t launch_down_fp8(const moe_grouped_fp8_desc& d, const void* h, const float* hs,
                           const int32_t* offsets, const int32_t* counts, const void* w2,
                           const float* s2, void* y, hipStream_t s) {
  Fp8Args g = operands(h, hs, w2, s2, d.inner, d.cols);
  g.offsets = offsets, g.counts = counts, g.groups = d.num_groups;
  g.m_cap = d.m_cap, g.max_rows = static_cast<int>(std::min<int64_t>(d.max_rows, INT32_MAX));
  g.e.out = y, g.e.ldo = d.cols, g.e.vec = true;
  if (d.fast) return launch8<kGrouped, 256, 256, 2>(g, INT64_MAX, s);
  return launch8<kGrouped, kExactRows, 256, 2, true>(g, INT64_MAX, s);
}

}  // namespace moe
