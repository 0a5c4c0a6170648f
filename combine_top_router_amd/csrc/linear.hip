// Dense matrix product with bias, activation and residual in its epilogue,
// and its gradients, on the matrix cores.
//
//   forward   z = x w^T + bias,  y = act(z) + residual      (x [M, K], w N x K)
//   backward  dz = dy act'(z),   dx = dz w,  dw = dz^T x,  dbias = column sums of dz
//
// All three products are one kernel, C[m, n] = sum_k A(m, k) B(n, k), with
// each operand in one of two memory forms:
//   by rows      (m, k) at m*ld + k: the reduction index is contiguous
//   by columns   (m, k) at k*ld + m: the output index is contiguous
// The forward reads x by rows and w by rows ([N, K]) or by columns ([K, N]);
// dx reads dz by rows and w the other way round; dw reads both by columns.
//
//  * dz is an fp32 value (dy act' or an fp32 dy), and the matrix cores read
//    16-bit ones: it goes in as two, dz = hi + lo with hi = dz rounded and lo
//    the rest rounded (2^-16 of dz left out in bf16, 2^-22 in fp16), whose
//    products are summed together. One 16-bit part alone, at the caller's wish,
//    gives dx and dw a second rounding (2.4e-3 of their norm instead of 1.7e-3
//    in bf16) and halves the products.
//  * v_mfma_f32_32x32x16: a lane feeds 8 consecutive k of one row of A and of
//    B. By-rows tiles give them as one 16-byte LDS read; by-columns tiles lie
//    in LDS as in memory and are transposed on the way out
//    (ds_read_b64_tr_b16, two reads of 4 rows x 16 columns).
//  * Tiles go memory -> LDS without registers (buffer_load ... lds) through a
//    ring of NS slices of 64 k, one barrier a slice, placed before the slice's
//    last step: that step's products run on fragments already read while the
//    next slice's first fragments and the loads of slice kt+NS go out, one
//    each behind a product. The 16-byte chunks of a row are XOR-swizzled so
//    that the reads cover the LDS banks (no bank conflicts counted).
//  * Rows past an operand's end, chunks past the end of the reduction and
//    slices past a split's end are given offsets beyond the buffer range: they
//    read as zeros, so the loop has one form and the counted waits stay exact.
//  * Bound, at 4096x14336x4096 (349 us, 1380 TFLOP/s): the matrix pipes are
//    busy 74 % of the cycles at the 1.66 GHz the chip holds under this load.
//  * Few output tiles and a long reduction: the slices are split over several
//    workgroups, each stores its fp32 sums, and a second launch adds them in
//    order and does the epilogue (results do not depend on timing).
//  * Products of 16-bit values are exact in fp32 and summed in fp32; the
//    epilogue is fp32, with one rounding per stored value.
#include <algorithm>
#include <iterator>

#include "linear_gemm.h"

namespace moe {
namespace {

// dz = dy act'(pre), in one or two parts of the rows' type, each padded to nw
// columns (zeros past N), and the column sums of the unrounded dz over this block's rows.
// A thread owns eight columns; a block 8 row lanes x 32 column groups.
struct ActGradArgs {
  const void* dy;
  const uint16_t* pre;  // or nullptr: dz = dy
  uint16_t* dz;         // or nullptr
  float* sums;          // [gridDim.y, nw] or nullptr
  int64_t ldy, ldp, ldz, nw, M;
  int part;             // columns from dz's first part to its second, or 0: one part
  int N, act, rows_per_block;
  bool f16, dy_f32, vec;  // vec: rows of dy and pre start 16-byte aligned
};

__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  __shared__ float red[8][32][8];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n = (int(blockIdx.x) * 32 + cx) * 8;
  const int64_t r0 = int64_t(blockIdx.y) * a.rows_per_block;
  const int64_t r1 = min(a.M, r0 + a.rows_per_block);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n < a.N) {
    const int cols = min(8, a.N - n);
    // dz of row m, its sums and its store
    auto finish = [&](int64_t m, float (&d)[8], const float (&z)[8]) __attribute__((always_inline)) {
      if (a.pre) {
        switch (a.act) {  // one uniform branch for the eight
          case MOE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= act_slope(z[i], MOE_ACT_RELU);
            break;
          case MOE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= act_slope(z[i], MOE_ACT_SILU);
            break;
          default:
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= act_slope(z[i], MOE_ACT_GELU);
            break;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = i < cols ? d[i] : 0.f;
        sum[i] += d[i];
      }
      if (!a.dz) return;
      const u32x4 hi = pack8x16(d, a.f16);
      *reinterpret_cast<u32x4*>(a.dz + m * a.ldz + n) = hi;
      if (!a.part) return;
      float h[8];
      unpack8x16(hi, h, a.f16);
#pragma unroll
      for (int i = 0; i < 8; ++i)  // (nothing beside an infinite part: inf - inf is NaN)
        h[i] = fabsf(h[i]) == INFINITY ? 0.f : d[i] - h[i];
      *reinterpret_cast<u32x4*>(a.dz + m * a.ldz + a.part + n) = pack8x16(h, a.f16);
    };
    if (a.vec && cols == 8) {
      constexpr int kRows = 2;  // rows whose loads are in flight together
      for (int64_t m0 = r0 + ry; m0 < r1; m0 += 8 * kRows) {
        u32x4 x[kRows], y[kRows], p[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int64_t m = m0 + 8 * u;
          if (m >= r1) continue;
          const char* at = static_cast<const char*>(a.dy) + (m * a.ldy + n) * (a.dy_f32 ? 4 : 2);
          x[u] = *reinterpret_cast<const u32x4*>(at);
          if (a.dy_f32) y[u] = *reinterpret_cast<const u32x4*>(at + 16);
          if (a.pre) p[u] = load8x16(a.pre + m * a.ldp + n);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int64_t m = m0 + 8 * u;
          if (m >= r1) continue;
          float d[8], z[8];
          if (a.dy_f32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              d[i] = __uint_as_float(x[u][i]), d[4 + i] = __uint_as_float(y[u][i]);
          } else {
            unpack8x16(x[u], d, a.f16);
          }
          if (a.pre) unpack8x16(p[u], z, a.f16);
          finish(m, d, z);
        }
      }
    } else {
      for (int64_t m = r0 + ry; m < r1; m += 8) {
        float d[8], z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = i < cols;
          d[i] = !in ? 0.f
                     : a.dy_f32 ? static_cast<const float*>(a.dy)[m * a.ldy + n + i]
                                : from16(static_cast<const uint16_t*>(a.dy)[m * a.ldy + n + i], a.f16);
          z[i] = in && a.pre ? from16(a.pre[m * a.ldp + n + i], a.f16) : 0.f;
        }
        finish(m, d, z);
      }
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[ry][cx][i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x >> 3, i = threadIdx.x & 7;
  float s = 0.f;
#pragma unroll
  for (int r = 0; r < 8; ++r) s += red[r][c][i];
  const int col = (int(blockIdx.x) * 32 + c) * 8 + i;
  if (col < a.nw) a.sums[int64_t(blockIdx.y) * a.nw + col] = s;
}

// dbias[n] = the blocks' column sums, added in order in fp64: 64 columns to a
// workgroup, each of its four wavefronts a quarter of the blocks.
__global__ __launch_bounds__(256) void bias_grad_kernel(const float* sums, int blocks, int64_t nw,
                                                        int N, float* dbias) {
  __shared__ double part[4][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int n = int(blockIdx.x) * 64 + c;
  const int per = (blocks + 3) / 4, b0 = q * per, b1 = min(blocks, b0 + per);
  double s = 0.0;
  if (n < N) {
    constexpr int kBatch = 8;  // loads in flight together
    for (int b = b0; b < b1; b += kBatch) {
      float x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) x[u] = b + u < b1 ? sums[(b + u) * nw + n] : 0.f;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) s += double(x[u]);
    }
  }
  part[q][c] = s;
  __syncthreads();
  if (q == 0 && n < N)
    dbias[n] = static_cast<float>(part[0][c] + part[1][c] + part[2][c] + part[3][c]);
}

// ---- host

constexpr int BK = 64;  // reduction indexes of a slice

// A tile shape with what its workgroups take, in microseconds: a slice on a
// quiet chip, a slice where a second workgroup shares the compute unit (per_cu
// 2), and a workgroup's beginning and end without its stores.
struct Tile {
  int bm, bn, threads, per_cu;
  double slice, shared, fixed;
};
constexpr Tile kTiles[] = {
    {256, 256, 512, 1, 0.87, 0.0, 2.5},   {128, 256, 512, 1, 0.55, 0.0, 2.9},
    {128, 128, 256, 2, 0.45, 1.35, 2.4},  {64, 128, 256, 2, 0.30, 0.89, 2.4},
    {64, 64, 256, 2, 0.225, 0.59, 2.0},   {128, 128, 512, 1, 0.375, 0.0, 2.5},
};
constexpr int64_t kLaunchThreads = (int64_t(1) << 32) - 1;
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128};

struct Plan {
  int tile, splits, per_split, halved;
  int64_t part_bytes;
};

// Tile and split of one product, from its sizes alone: the least estimated
// time. Rounds of workgroups over the chip, each of its slices (slower the
// more of the chip works: clock and memory) and its stores; at least
// the memory's time for the operands; for a split the second launch. The
// figures are a fit to 25000 timings of these tiles and splits on 800
// products of 1 to 65536 rows and 8 to 16384 columns and terms; on them the choice is 1.1 % slower
// than the best on average and 25 % at worst. Examples: 4096x14336x4096 takes
// 256x256 (349 us, 128x128 402-457 us), 16x7168x256 64x64 in 16 parts (9 us;
// whole, 34 us), 8192x256x7168 128x128 (57 us, 256x256 70 us).
Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t cus) {
  const int64_t all = std::max<int64_t>(1, (K + BK - 1) / BK);
  const int64_t nw = (N + 7) / 8 * 8;
  const double mem = (double(M) * K + double(N) * K + double(M) * N) * 2.0 / 5.75e6;
  Plan best{0, 1, static_cast<int>(all), 0, 0};
  double best_t = 1e300;
  for (int t = 0; t < int(std::size(kTiles)); ++t) {
    const Tile& c = kTiles[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (const int want : kSplits) {
      if (want > 1 && want * 2 > all) break;
      const int64_t per = (all + want - 1) / want, s = (all + per - 1) / per, groups = tiles * s;
      // what the launches take (cus: the most tiles that are halved)
      if ((groups + cus) * c.threads > kLaunchThreads || (s > 1 && M * nw / 8 + 64 > kLaunchThreads)) break;
      const double out = double(std::min<int64_t>(c.bm, M)) * double(std::min<int64_t>(c.bn, N)) *
                         (s > 1 ? 4.0 : 2.0) / 3.45e6;  // one workgroup's stores, us
      const int64_t slots = cus * c.per_cu, full = groups / slots, rest = groups % slots;
      const double load = double(rest) / double(cus), p = double(per);
      double time;
      int halved = 0;
      if (c.per_cu == 1) {
        const double round = p * c.slice * 1.7 + c.fixed + double(cus) * out;
        time = double(full) * round;
        // A last round that fills at most half of an XCD's compute units: its tiles
        // are cut in two (8192x2048x7168, 3.5 rounds: 230 -> 218 us).
        const int64_t last = groups / 8 % (cus / 8) + (groups % 8 ? 1 : 0);
        if (t == 0 && s == 1 && full > 0 && rest > 0 && last <= cus / 16)
          halved = static_cast<int>(last), time += 0.83 * round;
        else if (rest > 0)
          time += p * c.slice * (1.0 + 0.7 * load) + c.fixed + double(rest) * out;
      } else {
        time = double(full) * (std::max(p * c.shared, double(slots) * out) + c.fixed);
        if (rest > cus)
          time += p * c.shared * (1.0 - 0.25 * (2.0 - load)) + c.fixed + 0.5 * double(rest) * out;
        else if (rest > 0)
          time += p * c.slice * (1.0 + 0.5 * load) + c.fixed + double(rest) * out;
      }
      time = std::max(time, mem);
      if (s > 1) time += 1.4 + 0.07 * double(s) + double(s) * double(M) * double(nw) * 4.0 / 5.4e6;
      if (time < best_t) {
        best_t = time;
        best = {t, static_cast<int>(s), static_cast<int>(per), halved, s > 1 ? s * M * nw * 4 : 0};
      }
    }
  }
  return best;
}

// The last few plans of this thread: a call asks for its plan several times over
// (its workspace, the check of it, the launch), and making one takes 2 us.
Plan plan_product(int64_t M, int64_t N, int64_t K) {
  struct Known {
    int64_t M, N, K, cus;
    Plan p;
  };
  constexpr int kKnown = 16;
  thread_local Known known[kKnown] = {};
  thread_local int next = 0;
  const int64_t cus = device_cu_count();
  for (const Known& k : known)
    if (k.cus == cus && k.M == M && k.N == N && k.K == K) return k.p;
  const Plan p = make_plan(M, N, K, cus);
  known[next] = {M, N, K, cus, p};
  next = (next + 1) % kKnown;
  return p;
}

// Whether a product's launch has fewer than 2^32 threads: false where no tile's would.
bool launchable(int64_t M, int64_t N, int64_t K) {
  const Plan p = plan_product(M, N, K);
  const Tile& c = kTiles[p.tile];
  const int64_t groups =
      ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn) * p.splits + 8 * p.halved;
  return groups * c.threads <= kLaunchThreads;
}

template <bool F16, bool AC, bool BC>
void launch_product(const GemmArgs& g, int tile, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(int64_t(g.tiles_m) * g.tiles_n * g.splits + 8 * g.halved));
  switch (tile) {
    case 0: linear_kernel<F16, AC, BC, 256, 256, BK, 2, 4, 2, 2><<<grid, 512, 0, s>>>(g); break;
    case 1: linear_kernel<F16, AC, BC, 128, 256, BK, 2, 4, 3, 2><<<grid, 512, 0, s>>>(g); break;
    case 2: linear_kernel<F16, AC, BC, 128, 128, BK, 2, 2, 2, 2><<<grid, 256, 0, s>>>(g); break;
    case 3: linear_kernel<F16, AC, BC, 64, 128, BK, 1, 4, 3, 2><<<grid, 256, 0, s>>>(g); break;
    case 4: linear_kernel<F16, AC, BC, 64, 64, BK, 2, 2, 4, 2><<<grid, 256, 0, s>>>(g); break;
    default: linear_kernel<F16, AC, BC, 128, 128, BK, 2, 4, 4, 2><<<grid, 512, 0, s>>>(g); break;
  }
}

// The reduction of a product with an operand in two parts.
int64_t two_parts(int64_t K) { return 2 * ((K + BK - 1) / BK * BK); }

hipError_t product(GemmArgs g, bool a_cols, bool b_cols, void* ws, hipStream_t s) {
  if (g.M == 0 || g.N == 0) return hipSuccess;
  const Plan p = plan_product(g.M, g.N, g.two ? two_parts(g.K) : g.K);
  const Tile& c = kTiles[p.tile];
  g.tiles_m = static_cast<int>((g.M + c.bm - 1) / c.bm);
  g.tiles_n = static_cast<int>((g.N + c.bn - 1) / c.bn);
  g.splits = p.splits, g.per_split = p.per_split, g.halved = p.halved;
  g.part = static_cast<float*>(ws), g.nw = (g.N + 7) / 8 * 8;
  if (g.e.f16) {
    if (a_cols) launch_product<true, true, true>(g, p.tile, s);
    else if (b_cols) launch_product<true, false, true>(g, p.tile, s);
    else launch_product<true, false, false>(g, p.tile, s);
  } else {
    if (a_cols) launch_product<false, true, true>(g, p.tile, s);
    else if (b_cols) launch_product<false, false, true>(g, p.tile, s);
    else launch_product<false, false, false>(g, p.tile, s);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || g.splits == 1) return err;
  const int64_t threads = g.M * (g.nw / 8);
  linear_join_kernel<<<dim3(static_cast<unsigned>((threads + 63) / 64)), 64, 0, s>>>(g);
  return hipGetLastError();
}

bool aligned(const void* p, int64_t ld_bytes) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld_bytes & 15) == 0);
}

int act_kind(const moe_linear_desc& d) { return d.act & ~MOE_DZ_16BIT; }

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

// the backward's own buffers, in order: dz, the blocks' column sums, the splits' sums
struct BackwardPlan {
  int64_t nw, dz_bytes, sums_bytes, part_bytes;
  int row_blocks, rows_per_block;
};

// The workspace has to be known before the buffers are, so it always has room for
// dz in two parts and for the splits of either product.
BackwardPlan plan_backward(const moe_linear_desc& d) {
  BackwardPlan p{};
  const int64_t M = d.rows, N = d.cols, K = d.inner;
  p.nw = (N + 7) / 8 * 8;
  p.dz_bytes = round256(M * 2 * p.nw * 2);
  // about sixteen workgroups of 256 columns to a compute unit, 8 rows at least
  const int64_t cols = (N + 255) / 256;
  const int64_t want = std::max<int64_t>(1, 16 * device_cu_count() / cols);
  p.rows_per_block = static_cast<int>(std::max<int64_t>(8, ((M + want - 1) / want + 7) / 8 * 8));
  p.row_blocks = static_cast<int>((M + p.rows_per_block - 1) / p.rows_per_block);
  p.sums_bytes = round256(int64_t(p.row_blocks) * p.nw * 4);
  const bool nk = d.w_order == MOE_W_NK;
  const int64_t a = nk ? N : K, b = nk ? K : N;  // dw's rows and columns
  p.part_bytes = std::max({plan_product(M, K, N).part_bytes, plan_product(M, K, two_parts(N)).part_bytes,
                           plan_product(a, b, M).part_bytes, plan_product(a, b, two_parts(M)).part_bytes});
  return p;
}

}  // namespace

bool linear_launchable(const moe_linear_desc& d) { return launchable(d.rows, d.cols, d.inner); }

bool linear_backward_launchable(const moe_linear_desc& d) {
  const int64_t M = d.rows, N = d.cols, K = d.inner;
  const bool nk = d.w_order == MOE_W_NK;
  const int64_t a = nk ? N : K, b = nk ? K : N;  // dw's rows and columns
  return launchable(M, K, N) && launchable(M, K, two_parts(N)) && launchable(a, b, M) &&
         launchable(a, b, two_parts(M));
}

size_t linear_workspace_bytes(const moe_linear_desc& d) {
  return static_cast<size_t>(plan_product(d.rows, d.cols, d.inner).part_bytes);
}

size_t linear_backward_workspace_bytes(const moe_linear_desc& d) {
  const BackwardPlan p = plan_backward(d);
  return static_cast<size_t>(p.dz_bytes + p.sums_bytes + p.part_bytes);
}

hipError_t launch_linear(const moe_linear_desc& d, const void* x, const void* w,
                         const float* bias, const void* residual, void* y, void* pre, void* ws,
                         hipStream_t s) {
  GemmArgs g{};
  g.a = static_cast<const uint16_t*>(x), g.b = static_cast<const uint16_t*>(w);
  g.lda = d.ldx, g.ldb = d.ldw;
  g.M = d.rows, g.N = d.cols, g.K = d.inner;
  const bool nk = d.w_order == MOE_W_NK;
  g.a_ext = d.inner, g.b_ext = nk ? d.inner : d.cols;
  g.e.out = y, g.e.bias = bias;
  g.e.res = static_cast<const uint16_t*>(residual), g.e.pre = static_cast<uint16_t*>(pre);
  g.e.ldo = d.ldy, g.e.ldr = d.ldr, g.e.ldp = d.ldp;
  g.e.act = act_kind(d), g.e.f16 = d.dtype == MOE_ROWS_F16, g.e.out_f32 = d.y_f32 != 0;
  g.e.vec = aligned(y, d.ldy * (d.y_f32 ? 4 : 2)) && aligned(residual, d.ldr * 2) &&
            aligned(pre, d.ldp * 2);
  return product(g, false, !nk, ws, s);
}

hipError_t launch_linear_backward(const moe_linear_desc& d, const void* dy, const void* x,
                                  const void* w, const void* pre, void* dx, void* dw,
                                  float* dbias, void* ws, hipStream_t s) {
  const BackwardPlan p = plan_backward(d);
  char* at = static_cast<char*>(ws);
  uint16_t* dz = reinterpret_cast<uint16_t*>(at);
  float* sums = reinterpret_cast<float*>(at + p.dz_bytes);
  void* part = at + p.dz_bytes + p.sums_bytes;
  const int64_t M = d.rows;
  const int N = d.cols, K = d.inner;
  const int act = act_kind(d);
  const bool f16 = d.dtype == MOE_ROWS_F16, nk = d.w_order == MOE_W_NK;
  // dy is dz itself where nothing is to be done to it and its rows can be loaded as they are
  const bool copy = (dx || dw) && (act != MOE_ACT_NONE || d.y_f32 || N % 8 || !aligned(dy, d.ldy * 2));
  // one part holds a 16-bit dy, and what relu leaves of it
  const bool two = copy && !(d.act & MOE_DZ_16BIT) &&
                   (d.y_f32 || act == MOE_ACT_SILU || act == MOE_ACT_GELU);
  const int lo = two ? static_cast<int>(p.nw) : 0;  // where dz's second part begins
  const int64_t ldz = copy ? p.nw + lo : d.ldy;
  if (M > 0 && (copy || dbias)) {
    ActGradArgs a{};
    a.dy = dy, a.pre = act != MOE_ACT_NONE ? static_cast<const uint16_t*>(pre) : nullptr;
    a.dz = copy ? dz : nullptr, a.sums = dbias ? sums : nullptr;
    a.ldy = d.ldy, a.ldp = d.ldp, a.ldz = ldz, a.nw = p.nw, a.M = M;
    a.part = lo, a.N = N, a.act = act, a.rows_per_block = p.rows_per_block;
    a.f16 = f16, a.dy_f32 = d.y_f32 != 0;
    a.vec = aligned(dy, d.ldy * (d.y_f32 ? 4 : 2)) && aligned(a.pre, d.ldp * 2);
    act_grad_kernel<<<dim3((N + 255) / 256, p.row_blocks), 256, 0, s>>>(a);
    if (hipError_t err = hipGetLastError()) return err;
  }
  if (dbias) {
    bias_grad_kernel<<<dim3((N + 63) / 64), 256, 0, s>>>(sums, p.row_blocks, p.nw, N, dbias);
    if (hipError_t err = hipGetLastError()) return err;
  }
  const uint16_t* z = copy ? dz : static_cast<const uint16_t*>(dy);
  const int z_ext = static_cast<int>(p.nw);  // N, or N with its zeros
  GemmArgs g{};
  g.e.f16 = f16, g.e.act = MOE_ACT_NONE, g.two = two ? 1 : 0;
  if (dx) {  // dx[m, k] = sum_n dz[m, n] w[n, k]
    g.a = z, g.lda = ldz, g.a_ext = z_ext, g.a_part = lo;
    g.b = static_cast<const uint16_t*>(w), g.ldb = d.ldw, g.b_ext = nk ? K : N;
    g.M = M, g.N = K, g.K = N;
    g.e.out = dx, g.e.ldo = K;
    g.e.vec = aligned(dx, int64_t(K) * 2);
    if (hipError_t err = product(g, false, nk, part, s)) return err;
  }
  if (dw) {
    const uint16_t* xs = static_cast<const uint16_t*>(x);
    g.K = M;
    if (nk) {  // dw[n, k] = sum_m dz[m, n] x[m, k]
      g.a = z, g.lda = ldz, g.a_ext = z_ext, g.a_part = lo, g.M = N;
      g.b = xs, g.ldb = d.ldx, g.b_ext = K, g.b_part = 0, g.N = K;
    } else {   // dw[k, n] = sum_m x[m, k] dz[m, n]
      g.a = xs, g.lda = d.ldx, g.a_ext = K, g.a_part = 0, g.M = K;
      g.b = z, g.ldb = ldz, g.b_ext = z_ext, g.b_part = lo, g.N = N;
    }
    g.e.out = dw, g.e.ldo = g.N;
    g.e.vec = aligned(dw, g.N * 2);
    if (hipError_t err = product(g, true, true, part, s)) return err;
  }
  return hipSuccess;
}

}  // namespace moe
