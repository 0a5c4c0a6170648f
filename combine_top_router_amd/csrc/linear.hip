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
//  * v_mfma_f32_32x32x16: a lane feeds 8 consecutive k of one row of A and of
//    B. By-rows tiles give them as one 16-byte LDS read; by-columns tiles lie
//    in LDS as in memory and are transposed on the way out
//    (ds_read_b64_tr_b16, two reads of 4 rows x 16 columns).
//  * Tiles go memory -> LDS without registers (buffer_load ... lds) through a
//    ring of NS slices of 64 k, one barrier a slice. The 16-byte chunks of a
//    row are XOR-swizzled so that the reads cover the LDS banks.
//  * Rows past an operand's end, and the chunks past the end of the reduction,
//    are given offsets beyond the buffer range: they read as zeros.
//  * Few output tiles and a long reduction: the slices are split over several
//    workgroups, each stores its fp32 sums, and a second launch adds them in
//    order and does the epilogue (results do not depend on timing).
//  * Products of 16-bit values are exact in fp32 and summed in fp32; the
//    epilogue is fp32, with one rounding per stored value.
#include <algorithm>

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int BK = 64;  // reduction indexes of a slice

// A byte offset past every buffer range (a tile's range is at most 256 rows of
// 2^21 elements, 2^30 bytes), with room for a slice's advance on top.
constexpr uint32_t kOutside = 0x80000000u;

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

struct Epilogue {
  void* out;            // [M, N], ldo apart: 16-bit rows or fp32
  const float* bias;    // [N] or nullptr
  const uint16_t* res;  // [M, N] or nullptr
  uint16_t* pre;        // [M, N] or nullptr: receives z
  int64_t ldo, ldr, ldp;
  int act;
  bool f16, out_f32;
  bool vec;  // every row of out, res and pre starts 16-byte aligned
};

struct GemmArgs {
  const uint16_t* a;
  const uint16_t* b;
  int64_t lda, ldb;     // elements
  int64_t M, N, K;      // output rows and columns, reduction
  int a_ext, b_ext;     // contiguous extent of an operand's rows (reduction or output index)
  int tiles_m, tiles_n;
  int splits, per_split;  // slices of a split
  float* part;          // splits > 1: [splits, M, nw] fp32
  int64_t nw;
  Epilogue e;
};

__device__ __forceinline__ float from16(uint16_t b, bool f16) {
  return f16 ? static_cast<float>(__builtin_bit_cast(_Float16, b)) : from_bf16(b);
}
__device__ __forceinline__ uint16_t to16(float f, bool f16) {
  return f16 ? __builtin_bit_cast(uint16_t, static_cast<_Float16>(f)) : to_bf16(f);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool f16) {
  if (!f16) return pack_bf16x2(lo, hi);
  f16x2 v;
  v[0] = static_cast<_Float16>(lo);
  v[1] = static_cast<_Float16>(hi);
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ u32x4 pack8x16(const float (&f)[8], bool f16) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack16(f[2 * i], f[2 * i + 1], f16);
  return v;
}
__device__ __forceinline__ void unpack8x16(const u32x4& v, float (&f)[8], bool f16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = from16(static_cast<uint16_t>(v[i] & 0xffffu), f16);
    f[2 * i + 1] = from16(static_cast<uint16_t>(v[i] >> 16), f16);
  }
}

__device__ __forceinline__ float act_of(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? z : z * 0.f;  // NaN stays NaN
    case MOE_ACT_SILU: return z / (1.f + expf(-z));
    // erfc, not 1 + erf: no cancellation in the negative tail
    case MOE_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACT_GELU:
      return 0.5f * erfcf(-0.70710678118654752f * z) +
             z * expf(-0.5f * z * z) * 0.39894228040143268f;
    default: return 1.f;
  }
}

// Columns n .. n+7 of output row m from their sums.
__device__ __forceinline__ void finish8(const Epilogue& e, int64_t m, int64_t n, int64_t N,
                                        float (&v)[8]) {
  if (e.vec && n + 8 <= N) {
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += e.bias[n + i];
    }
    if (e.pre) *reinterpret_cast<u32x4*>(e.pre + m * e.ldp + n) = pack8x16(v, e.f16);
    if (e.act != MOE_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_of(v[i], e.act);
    }
    if (e.res) {
      float r[8];
      unpack8x16(*reinterpret_cast<const u32x4*>(e.res + m * e.ldr + n), r, e.f16);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    if (e.out_f32) {
      float* o = static_cast<float*>(e.out) + m * e.ldo + n;
      *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(e.out) + m * e.ldo + n) =
          pack8x16(v, e.f16);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (n + i >= N) continue;
    float z = v[i];
    if (e.bias) z += e.bias[n + i];
    if (e.pre) e.pre[m * e.ldp + n + i] = to16(z, e.f16);
    z = act_of(z, e.act);
    if (e.res) z += from16(e.res[m * e.ldr + n + i], e.f16);
    if (e.out_f32) static_cast<float*>(e.out)[m * e.ldo + n + i] = z;
    else static_cast<uint16_t*>(e.out)[m * e.ldo + n + i] = to16(z, e.f16);
  }
}

// Swizzle of a by-rows slice (128-byte rows): as the 16 rows that one LDS
// cycle reads at one logical chunk must land on 16 different bank groups, and
// a row's parity already picks one half of the banks, the key is the next
// three row bits.
__device__ __forceinline__ int row_key(int row) { return (row >> 1) & 7; }

// Swizzle of a by-columns slice with CPR 16-byte chunks to a row: the transposed
// read's 32 lanes take 64 bytes of 4 consecutive rows, which have to lie in
// different quarters of the banks.
template <int CPR>
__device__ __forceinline__ int col_key(int k) {
  return CPR >= 16 ? (k & 3) << 2 : CPR == 8 ? ((k >> 1) & 1) << 2 : 0;
}

// One operand's tile: D output indexes x BK reduction indexes.
template <int D, bool COLS, int WAVES>
struct Operand {
  static constexpr int BYTES = D * BK * 2;
  static constexpr int CPR = COLS ? D / 8 : 8;  // chunks of an LDS row
  static constexpr int RPL = 64 / CPR;          // LDS rows of a 1 KiB wave-load
  static constexpr int LOADS = BYTES / 1024 / WAVES;
  static_assert(LOADS * 1024 * WAVES == BYTES && LOADS >= 1, "whole wave-loads");

  const uint16_t* base;
  int64_t ld;
  int ext, valid;   // by rows: reduction extent, output rows left; by columns: row extent
  int64_t K;        // reduction length
  int d0;           // by columns: first output index of the tile
  i32x4 rsrc;
  uint32_t off[LOADS];
  int chunk;        // by rows: this lane's logical chunk of a slice

  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int64_t first,
                                       int64_t count, int ext_, int64_t K_, int wid, int lane) {
    ld = ld_, ext = ext_, K = K_;
    if constexpr (COLS) {
      base = p;
      d0 = static_cast<int>(first);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (wid + WAVES * i) * RPL + lane / CPR;
        const int c = (lane % CPR) ^ col_key<CPR>(k);
        // a chunk past the row's extent would be another row's data: harmless, as it
        // only reaches outputs that are not stored, but the last row has nothing behind it
        off[i] = d0 + 8 * c < ext ? (uint32_t(k) * uint32_t(ld) + uint32_t(d0 + 8 * c)) * 2u
                                  : kOutside;
      }
    } else {
      base = p + first * ld;
      valid = static_cast<int>(min(int64_t(D), count - first));
      rsrc = make_rsrc(base, (uint32_t(valid - 1) * uint32_t(ld) + uint32_t(ext)) * 2u);
      const int r0 = wid * RPL + lane / CPR;
      chunk = (lane % CPR) ^ row_key(r0);  // the other wave-loads start 8 * WAVES rows on: same key
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = r0 + WAVES * RPL * i;
        off[i] = r < valid ? (uint32_t(r) * uint32_t(ld) + uint32_t(chunk * 8)) * 2u : kOutside;
      }
    }
  }

  // the buffer range of slice kt (by columns: the rows of the slice that exist)
  __device__ __forceinline__ i32x4 slice(int kt) const {
    if constexpr (!COLS) return rsrc;
    const int rows = static_cast<int>(min(int64_t(BK), K - int64_t(kt) * BK));
    return make_rsrc(base + int64_t(kt) * BK * ld, (uint32_t(rows - 1) * uint32_t(ld) + uint32_t(ext)) * 2u);
  }

  // wave-load i of slice kt into the operand's LDS part at `lds`
  __device__ __forceinline__ void load(int i, const i32x4& r, int kt, uint32_t lds,
                                       int wid) const {
    const uint32_t to = lds + (wid + WAVES * i) * 1024;
    if constexpr (COLS) {
      dma16(r, off[i], to);
    } else if ((kt + 1) * BK <= ext) {
      dma16(r, off[i], uint32_t(kt) * (BK * 2), to);
    } else {  // the last, partial slice: chunks past the reduction read zeros
      const bool in = int(kt) * BK + chunk * 8 < ext;
      dma16(r, in ? off[i] : kOutside, uint32_t(kt) * (BK * 2), to);
    }
  }

  // the 32-row block at output index d of the 16-wide step kk
  static __device__ __forceinline__ u32x4 fragment(const char* s, int kk, int d, int lane) {
    if constexpr (COLS) {
      const int grp = lane >> 4, fr = (lane >> 2) & 3, fq = lane & 3;
      const int k = kk * 16 + 8 * (grp >> 1) + fr;
      const int c = d + 16 * (grp & 1) + 4 * fq;
      // rows k and k + 4 have the same key
      const char* p = s + k * (D * 2) + 16 * ((c >> 3) ^ col_key<CPR>(k)) + 8 * (fq & 1);
      const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p);
      const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * (D * 2)));
      const v8i16 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(u32x4, v);
    } else {
      const int row = d + (lane & 31), ch = 2 * kk + (lane >> 5);
      return *reinterpret_cast<const u32x4*>(s + row * (BK * 2) + ((ch ^ row_key(row)) << 4));
    }
  }
};

template <bool F16>
__device__ __forceinline__ f32x16 mma(const u32x4& a, const u32x4& b, const f32x16& c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

constexpr int kBand = 4;  // row tiles walked together

template <bool F16, bool ACOLS, bool BCOLS, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_kernel(GemmArgs g) {
  constexpr int WAVES = WM * WN;
  using OpA = Operand<BM, ACOLS, WAVES>;
  using OpB = Operand<BN, BCOLS, WAVES>;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int STAGE = OpA::BYTES + OpB::BYTES, NL = OpA::LOADS + OpB::LOADS;
  constexpr int EP = 32 * TN * 32 * 4;  // a wavefront's epilogue block: 32 rows x 32 TN floats
  static_assert(TM * WM * 32 == BM && TN * WN * 32 == BN, "tile");
  static_assert(EP * WAVES <= NS * STAGE && (TN == 1 || TN == 2), "epilogue block");
  __shared__ __attribute__((aligned(1024))) char smem[NS * STAGE];

  const int tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;

  // Workgroups are dealt to the 8 XCDs in turn: each XCD takes a contiguous
  // range of tiles, so that neighbours share operands behind one L2. Tiles go
  // in bands of kBand row tiles, column tile major inside a band.
  const int G = gridDim.x;
  const int xcd = blockIdx.x & 7, q8 = G >> 3, r8 = G & 7;
  const int id = xcd * q8 + min(xcd, r8) + (int(blockIdx.x) >> 3);
  const int tiles = g.tiles_m * g.tiles_n;
  const int split = id / tiles, tile = id - split * tiles;
  int mt, nt;
  {
    const int full = g.tiles_m / kBand * kBand;
    if (tile < full * g.tiles_n) {
      const int band = tile / (kBand * g.tiles_n), r2 = tile % (kBand * g.tiles_n);
      nt = r2 / kBand;
      mt = band * kBand + r2 % kBand;
    } else {
      const int tail = g.tiles_m - full, r2 = tile - full * g.tiles_n;
      nt = r2 / tail;
      mt = full + r2 % tail;
    }
  }
  const int64_t m0 = int64_t(mt) * BM, n0 = int64_t(nt) * BN;

  OpA A;
  OpB B;
  A.init(g.a, g.lda, m0, g.M, g.a_ext, g.K, wid, lane);
  B.init(g.b, g.ldb, n0, g.N, g.b_ext, g.K, wid, lane);
  const int all = static_cast<int>((g.K + BK - 1) / BK);
  const int k0 = split * g.per_split, k1 = min(all, k0 + g.per_split);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));

  auto issue = [&](int kt) {
    const uint32_t at = lds0 + (kt - k0) % NS * STAGE;
    const i32x4 ra = A.slice(kt), rb = B.slice(kt);
#pragma unroll
    for (int i = 0; i < OpA::LOADS; ++i) A.load(i, ra, kt, at, wid);
#pragma unroll
    for (int i = 0; i < OpB::LOADS; ++i) B.load(i, rb, kt, at + OpA::BYTES, wid);
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (k0 + s < k1) issue(k0 + s);
  for (int kt = k0; kt < k1; ++kt) {
    // slice kt has landed when at most the later slices' loads are in flight
    if (kt + NS - 2 < k1) wait_vmcnt<(NS - 2) * NL>(); else wait_vmcnt<0>();
    __syncthreads();  // ... every wavefront's part of it, and slice kt-1 is read
    if (kt + NS - 1 < k1) issue(kt + NS - 1);
    const char* sa = smem + (kt - k0) % NS * STAGE;
    const char* sb = sa + OpA::BYTES;
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      u32x4 fa[TM], fb[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fb[j] = OpB::fragment(sb, kk, wn * (32 * TN) + j * 32, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
        fa[i] = OpA::fragment(sa, kk, wm * (32 * TM) + i * 32, lane);
      // B first: each block of acc holds the transposed output block, so four
      // consecutive accumulators are four consecutive columns of one row
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mma<F16>(fb[j], fa[i], acc[i][j]);
    }
  }
  __syncthreads();  // the stages are free

  // Epilogue, each wavefront by itself: a 32-row block goes to its own LDS
  // part as fp32 (chunks of four columns, swizzled by row), then eight
  // columns of a row per lane come back.
  char* ep = smem + wid * EP;
  constexpr int ECH = 8 * TN;  // 16-byte chunks of a block's row
  auto slot = [](int r, int c) {
    const int key = ECH >= 16 ? (r & 15) : ((r >> 1) & 7);
    return r * (ECH * 16) + ((c ^ key) << 4);
  };
  for_each_index([&](auto i_tag) {
    constexpr int i = decltype(i_tag)::value;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(ep + slot(lane & 31, j * 8 + 2 * q + (lane >> 5))) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    // one wavefront's LDS accesses complete in order; the fence keeps the compiler's
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    constexpr int C8 = 4 * TN;  // groups of eight columns
#pragma unroll
    for (int it = 0; it < 32 * C8 / 64; ++it) {
      const int c = it * 64 + lane, r = c / C8, c8 = c % C8;
      const f32x4 x = *reinterpret_cast<const f32x4*>(ep + slot(r, 2 * c8));
      const f32x4 y = *reinterpret_cast<const f32x4*>(ep + slot(r, 2 * c8 + 1));
      float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      const int64_t m = m0 + wm * (32 * TM) + i * 32 + r;
      const int64_t n = n0 + wn * (32 * TN) + c8 * 8;
      if (m < g.M && n < g.N) {
        if (g.splits > 1) {
          float* p = g.part + (int64_t(split) * g.M + m) * g.nw + n;
          *reinterpret_cast<f32x4*>(p) = x;
          *reinterpret_cast<f32x4*>(p + 4) = y;
        } else {
          finish8(g.e, m, n, g.N, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }, std::make_integer_sequence<int, TM>{});
}

// The sums of the splits, in order, and the epilogue: eight columns a thread.
__global__ __launch_bounds__(256) void linear_join_kernel(GemmArgs g) {
  const int64_t c8 = g.nw / 8;
  const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (at >= g.M * c8) return;
  const int64_t m = at / c8, n = (at - m * c8) * 8;
  const float* p = g.part + m * g.nw + n;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.splits; ++s) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(p);
    const f32x4 y = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i], v[4 + i] += y[i];
    p += g.M * g.nw;
  }
  finish8(g.e, m, n, g.N, v);
}

// dz = dy act'(pre), rounded to the rows' type with its rows padded to ldz (zeros
// past N), and the column sums of the unrounded dz over this block's rows.
// A thread owns eight columns; a block 8 row lanes x 32 column groups.
struct ActGradArgs {
  const void* dy;
  const uint16_t* pre;  // or nullptr: dz = dy
  uint16_t* dz;         // or nullptr
  float* sums;          // [gridDim.y, nw] or nullptr
  int64_t ldy, ldp, ldz, nw, M;
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
    const bool full = a.vec && n + 8 <= a.N;
    for (int64_t m = r0 + ry; m < r1; m += 8) {
      float d[8], z[8];
      if (full) {
        if (a.dy_f32) {
          const float* p = static_cast<const float*>(a.dy) + m * a.ldy + n;
          const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = x[i], d[4 + i] = y[i];
        } else {
          unpack8x16(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.dy) + m * a.ldy + n),
                     d, a.f16);
        }
        if (a.pre) unpack8x16(*reinterpret_cast<const u32x4*>(a.pre + m * a.ldp + n), z, a.f16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = n + i < a.N;
          d[i] = !in ? 0.f
                     : a.dy_f32 ? static_cast<const float*>(a.dy)[m * a.ldy + n + i]
                                : from16(static_cast<const uint16_t*>(a.dy)[m * a.ldy + n + i], a.f16);
          z[i] = in && a.pre ? from16(a.pre[m * a.ldp + n + i], a.f16) : 0.f;
        }
      }
      if (a.pre) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < a.N) d[i] *= act_slope(z[i], a.act);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
      if (a.dz) *reinterpret_cast<u32x4*>(a.dz + m * a.ldz + n) = pack8x16(d, a.f16);
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

// dbias[n] = the blocks' column sums, added in order in fp64
__global__ __launch_bounds__(256) void bias_grad_kernel(const float* sums, int blocks, int64_t nw,
                                                        int N, float* dbias) {
  const int n = int(blockIdx.x) * 256 + threadIdx.x;
  if (n >= N) return;
  double s = 0.0;
  for (int b = 0; b < blocks; ++b) s += double(sums[b * nw + n]);
  dbias[n] = static_cast<float>(s);
}

// ---- host

struct Tile { int bm, bn; };
constexpr Tile kTiles[] = {{256, 256}, {128, 128}, {32, 128}, {128, 32}};

struct Plan {
  int tile, splits, per_split;
  int64_t part_bytes;
};

// Tile and split of one product, from its sizes alone.
Plan plan_product(int64_t M, int64_t N, int64_t K) {
  const int cus = device_cu_count();
  const int64_t all = (K + BK - 1) / BK;
  // workgroups a compute unit holds, and the time of a slice and of a
  // workgroup's beginning and end, in microseconds
  constexpr int per_cu[] = {1, 2, 2, 2};
  constexpr double slice[] = {1.9, 1.0, 0.45, 0.45}, fixed[] = {6.0, 4.0, 3.0, 3.0};
  Plan best{0, 1, static_cast<int>(all), 0};
  double best_t = 1e30;
  for (int t = 0; t < 4; ++t) {
    const int64_t tiles = ((M + kTiles[t].bm - 1) / kTiles[t].bm) *
                          ((N + kTiles[t].bn - 1) / kTiles[t].bn);
    for (int want = 1; want <= 128; want *= 2) {
      const int64_t per = (all + want - 1) / want;
      const int64_t s = per ? (all + per - 1) / per : 1;
      if (want > 1 && (s < 2 || per < 2)) break;
      const int64_t slots = int64_t(cus) * per_cu[t];
      const double rounds = double((tiles * s + slots - 1) / slots);
      double time = rounds * (double(per) * slice[t] + fixed[t]);
      if (s > 1) time += 4.0 + double(s) * double(M) * double(N) * 8.0 / 4e6;
      if (time < best_t) {
        best_t = time;
        best = {t, static_cast<int>(s), static_cast<int>(std::max<int64_t>(per, 1)),
                s > 1 ? s * M * ((N + 7) / 8 * 8) * 4 : 0};
      }
    }
  }
  return best;
}

template <bool F16, bool AC, bool BC>
void launch_product(const GemmArgs& g, int tile, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(int64_t(g.tiles_m) * g.tiles_n * g.splits));
  switch (tile) {
    case 0: linear_kernel<F16, AC, BC, 256, 256, 2, 4, 2><<<grid, 512, 0, s>>>(g); break;
    case 1: linear_kernel<F16, AC, BC, 128, 128, 2, 2, 2><<<grid, 256, 0, s>>>(g); break;
    case 2: linear_kernel<F16, AC, BC, 32, 128, 1, 4, 4><<<grid, 256, 0, s>>>(g); break;
    default: linear_kernel<F16, AC, BC, 128, 32, 4, 1, 4><<<grid, 256, 0, s>>>(g); break;
  }
}

hipError_t product(GemmArgs g, bool a_cols, bool b_cols, void* ws, hipStream_t s) {
  if (g.M == 0 || g.N == 0) return hipSuccess;
  const Plan p = plan_product(g.M, g.N, g.K);
  g.tiles_m = static_cast<int>((g.M + kTiles[p.tile].bm - 1) / kTiles[p.tile].bm);
  g.tiles_n = static_cast<int>((g.N + kTiles[p.tile].bn - 1) / kTiles[p.tile].bn);
  g.splits = p.splits, g.per_split = p.per_split;
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
  linear_join_kernel<<<dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, s>>>(g);
  return hipGetLastError();
}

bool aligned(const void* p, int64_t ld_bytes) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld_bytes & 15) == 0);
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

// the backward's own buffers, in order: dz, the blocks' column sums, the splits' sums
struct BackwardPlan {
  bool copy;  // dz is written (else dy serves as it is)
  int64_t ldz, dz_bytes, sums_bytes, part_bytes;
  int row_blocks, rows_per_block;
};

// The workspace has to be known before the buffers are, so it always has room for dz.
BackwardPlan plan_backward(const moe_linear_desc& d) {
  BackwardPlan p{};
  const int64_t M = d.rows, N = d.cols, K = d.inner;
  p.ldz = (N + 7) / 8 * 8;
  p.dz_bytes = round256(M * p.ldz * 2);
  // about four workgroups of 256 columns to a compute unit, 8 rows at least
  const int64_t cols = (N + 255) / 256;
  const int64_t want = std::max<int64_t>(1, 4 * device_cu_count() / cols);
  p.rows_per_block = static_cast<int>(std::max<int64_t>(8, ((M + want - 1) / want + 7) / 8 * 8));
  p.row_blocks = static_cast<int>((M + p.rows_per_block - 1) / p.rows_per_block);
  p.sums_bytes = round256(int64_t(p.row_blocks) * p.ldz * 4);
  const bool nk = d.w_order == MOE_W_NK;
  p.part_bytes = std::max(plan_product(M, K, N).part_bytes,
                          (nk ? plan_product(N, K, M) : plan_product(K, N, M)).part_bytes);
  return p;
}

}  // namespace

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
  g.e.act = d.act, g.e.f16 = d.dtype == MOE_ROWS_F16, g.e.out_f32 = d.y_f32 != 0;
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
  const bool f16 = d.dtype == MOE_ROWS_F16, act = d.act != MOE_ACT_NONE, nk = d.w_order == MOE_W_NK;
  // dy is dz itself where nothing is to be done to it and its rows can be loaded as they are
  const bool copy = (dx || dw) && (act || d.y_f32 || N % 8 || !aligned(dy, d.ldy * 2));
  if (M > 0 && (copy || dbias)) {
    ActGradArgs a{};
    a.dy = dy, a.pre = act ? static_cast<const uint16_t*>(pre) : nullptr;
    a.dz = copy ? dz : nullptr, a.sums = dbias ? sums : nullptr;
    a.ldy = d.ldy, a.ldp = d.ldp, a.ldz = p.ldz, a.nw = p.ldz, a.M = M;
    a.N = N, a.act = d.act, a.rows_per_block = p.rows_per_block;
    a.f16 = f16, a.dy_f32 = d.y_f32 != 0;
    a.vec = aligned(dy, d.ldy * (d.y_f32 ? 4 : 2)) && aligned(a.pre, d.ldp * 2);
    act_grad_kernel<<<dim3((N + 255) / 256, p.row_blocks), 256, 0, s>>>(a);
    if (hipError_t err = hipGetLastError()) return err;
  }
  if (dbias) {
    bias_grad_kernel<<<dim3((N + 255) / 256), 256, 0, s>>>(sums, p.row_blocks, p.ldz, N, dbias);
    if (hipError_t err = hipGetLastError()) return err;
  }
  const uint16_t* z = copy ? dz : static_cast<const uint16_t*>(dy);
  const int64_t ldz = copy ? p.ldz : d.ldy;
  const int z_ext = static_cast<int>(p.ldz);  // N, or N with its zeros
  GemmArgs g{};
  g.e.f16 = f16, g.e.act = MOE_ACT_NONE;
  if (dx) {  // dx[m, k] = sum_n dz[m, n] w[n, k]
    g.a = z, g.lda = ldz, g.a_ext = z_ext;
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
      g.a = z, g.lda = ldz, g.a_ext = z_ext, g.M = N;
      g.b = xs, g.ldb = d.ldx, g.b_ext = K, g.N = K;
    } else {   // dw[k, n] = sum_m x[m, k] dz[m, n]
      g.a = xs, g.lda = d.ldx, g.a_ext = K, g.M = K;
      g.b = z, g.ldb = ldz, g.b_ext = z_ext, g.N = N;
    }
    g.e.out = dw, g.e.ldo = g.N;
    g.e.vec = aligned(dw, g.N * 2);
    if (hipError_t err = product(g, true, true, part, s)) return err;
  }
  return hipSuccess;
}

}  // namespace moe
