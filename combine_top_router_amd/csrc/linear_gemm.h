// The tile kernel of the dense linear layer: C[m, n] = sum_k A(m, k) B(n, k)
// with the linear layer's epilogue (linear.hip has the whole picture).
#pragma once

#include "linear_epilogue.h"

namespace moe {
namespace {

// A byte offset past every buffer range (a tile's range is at most 256 rows of
// 2^21 elements, 2^30 bytes), with room for a slice's advance on top.
constexpr uint32_t kOutside = 0x80000000u;

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct GemmArgs {
  const uint16_t* a;
  const uint16_t* b;
  int64_t lda, ldb;     // elements
  int64_t M, N, K;      // output rows and columns, reduction
  int a_ext, b_ext;     // contiguous extent of an operand's rows (reduction or output index)
  int two;              // 1: each slice of the reduction comes twice, for an operand in two parts
  int a_part, b_part;   // where an operand's second part begins, from its first (0: the same again)
  int tiles_m, tiles_n;
  int splits, per_split;  // slices of a split
  int halved;             // tiles of each XCD that two workgroups share
  float* part;          // splits > 1: [splits, M, nw] fp32
  int64_t nw;
  Epilogue e;
};

// Swizzle of a by-rows slice: the 16 rows that one LDS cycle reads at one
// logical chunk must land on 16 different bank groups. A 128-byte row's parity
// already picks one half of the banks, so the key is the next three row bits.
__device__ __forceinline__ int row_key(int row) { return (row >> 1) & 7; }

// Swizzle of a by-columns slice with CPR 16-byte chunks to a row: the transposed
// read's 32 lanes take 64 bytes of 4 consecutive rows, which have to lie in
// different quarters of the banks.
template <int CPR>
__device__ __forceinline__ int col_key(int k) {
  static_assert(CPR >= 8, "64 columns or more");
  return CPR >= 16 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}

// One operand's tile: D output indexes x BK reduction indexes.
template <int D, int BK, bool COLS, int WAVES>
struct Operand {
  static constexpr int BYTES = D * BK * 2;
  static constexpr int CPR = COLS ? D / 8 : BK / 8;  // chunks of an LDS row
  static constexpr int RPL = 64 / CPR;          // LDS rows of a 1 KiB wave-load
  static constexpr int LOADS = BYTES / 1024 / WAVES;
  static_assert(LOADS * 1024 * WAVES == BYTES && LOADS >= 1, "whole wave-loads");
  static_assert(BK == 64, "row_key is that of 128-byte rows");

  const uint16_t* base;
  int64_t ld;
  int ext, valid;   // by rows: reduction extent, output rows left; by columns: row extent
  int64_t K;        // reduction length
  int two, part;    // GemmArgs
  int d0;           // by columns: first output index of the tile
  i32x4 rsrc;
  uint32_t off[LOADS];
  int chunk;        // by rows: this lane's logical chunk of a slice

  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int64_t first,
                                       int64_t count, int height, int ext_, int64_t K_, int two_,
                                       int part_, int wid, int lane) {
    ld = ld_, ext = ext_, K = K_, two = two_, part = part_;
    if constexpr (COLS) {
      base = p;
      d0 = static_cast<int>(first);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (wid + WAVES * i) * RPL + lane / CPR;
        const int c = (lane % CPR) ^ col_key<CPR>(k);
        // a chunk past the row's extent would be another row's data: harmless, as it
        // only reaches outputs that are not stored, but the last row has nothing behind it
        off[i] = d0 + 8 * c < ext && 8 * c < height ? (uint32_t(k) * uint32_t(ld) + uint32_t(d0 + 8 * c)) * 2u
                                  : kOutside;
      }
    } else {
      base = p + first * ld;
      valid = static_cast<int>(min(int64_t(height), count - first));
      rsrc = make_rsrc(base, (uint32_t(valid - 1) * uint32_t(ld) + uint32_t(part + ext)) * 2u);
      static_assert(WAVES * RPL % 32 == 0, "one key for all wave-loads");
      const int r0 = wid * RPL + lane / CPR;
      chunk = (lane % CPR) ^ row_key(r0);  // the other wave-loads start a multiple of 32 rows on: same key
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = r0 + WAVES * RPL * i;
        off[i] = r < valid ? (uint32_t(r) * uint32_t(ld) + uint32_t(chunk * 8)) * 2u : kOutside;
      }
    }
  }

  // Slice kt's loads: by columns, the buffer range ends with the slice's last row;
  // by rows, a chunk past the reduction's end gets an offset outside. Slices
  // from `end` on read nothing but zeros (so that the loop has no last rounds
  // of its own: such loads cost no memory traffic). With an operand in two parts,
  // slices 2 k and 2 k + 1 are those of its parts at reduction slice k, so that
  // the other operand's tile is read again while it is still in the caches.
  struct Slice {
    i32x4 rsrc;
    bool in;
    uint32_t advance;
  };
  __device__ __forceinline__ Slice slice(int kt, int end) const {
    Slice s;
    const int k = kt >> two, add = kt & two ? part : 0;
    if constexpr (COLS) {
      const int rows = kt < end ? static_cast<int>(min(int64_t(BK), K - int64_t(k) * BK)) : 0;
      s.rsrc = make_rsrc(base + (int64_t(k) * BK * ld + add),
                         rows ? (uint32_t(rows - 1) * uint32_t(ld) + uint32_t(ext)) * 2u : 0u);
      s.in = true, s.advance = 0;
    } else {
      s.rsrc = rsrc;
      s.in = kt < end && k * BK + chunk * 8 < ext;
      s.advance = uint32_t(k) * (BK * 2) + uint32_t(add) * 2u;
    }
    return s;
  }

  // wave-load i of a slice into the operand's LDS part at `lds`
  __device__ __forceinline__ void load(int i, const Slice& s, uint32_t lds, int wid) const {
    const uint32_t to = lds + (wid + WAVES * i) * 1024;
    if constexpr (COLS) dma16(s.rsrc, off[i], to);
    else dma16(s.rsrc, s.in ? off[i] : kOutside, s.advance, to);
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

// Scheduling of a step with NR fragment reads and NP products: the reads go
// between the products, two at a time from the first product on, so that the
// next step's fragments are there when its first product starts.
template <int T, int NR, int NP>
__device__ __forceinline__ void interleave_slot() {
  if constexpr (T < NP) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // product
    constexpr int PER = (NR + NP - 1) / NP;
    if constexpr (T * PER < NR)
      __builtin_amdgcn_sched_group_barrier(0x100, NR - T * PER < PER ? NR - T * PER : PER, 0);
    interleave_slot<T + 1, NR, NP>();
  }
}
template <int NR, int NP>
__device__ __forceinline__ void interleave() { interleave_slot<0, NR, NP>(); }

constexpr int kBand = 4;  // row tiles walked together

template <bool F16, bool ACOLS, bool BCOLS, int BM, int BN, int BK, int WM, int WN, int NS, int OCC>
__global__ __launch_bounds__(64 * WM * WN, OCC) void linear_kernel(GemmArgs g) {
  constexpr int WAVES = WM * WN;
  using OpA = Operand<BM, BK, ACOLS, WAVES>;
  using OpB = Operand<BN, BK, BCOLS, WAVES>;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32, KK = BK / 16;
  constexpr int STAGE = OpA::BYTES + OpB::BYTES, NL = OpA::LOADS + OpB::LOADS;
  constexpr int EP = 32 * TN * 32 * 4;  // a wavefront's epilogue block: 32 rows x 32 TN floats
  static_assert(TM * WM * 32 == BM && TN * WN * 32 == BN, "tile");
  static_assert(EP * WAVES <= NS * STAGE && (TN == 1 || TN == 2), "epilogue block");
  __shared__ __attribute__((aligned(1024))) char smem[NS * STAGE];

  const int tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;

  // Workgroups are dealt to the 8 XCDs in turn: each XCD takes a contiguous
  // range of tiles, so that neighbours share operands behind one L2. Tiles go
  // in bands of kBand row tiles, column tile major inside a band. The last
  // `halved` tiles of each XCD are two workgroups each, of half the rows.
  const int tiles = g.tiles_m * g.tiles_n;
  const int xcd = blockIdx.x & 7, nth = int(blockIdx.x) >> 3;
  const int ids = tiles * g.splits, q8 = ids >> 3, r8 = ids & 7;
  const int whole = q8 + (xcd < r8 ? 1 : 0) - g.halved;
  int id = xcd * q8 + min(xcd, r8), height = BM, half = 0;
  if (nth < whole) {
    id += nth;
  } else {
    id += whole + ((nth - whole) >> 1);
    half = (nth - whole) & 1, height = BM / 2;
  }
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
  const int64_t m0 = int64_t(mt) * BM + half * (BM / 2), n0 = int64_t(nt) * BN;
  if (m0 >= g.M) return;  // the lower half of a tile that has none

  OpA A;
  OpB B;
  A.init(g.a, g.lda, m0, g.M, height, g.a_ext, g.K, g.two, g.a_part, wid, lane);
  B.init(g.b, g.ldb, n0, g.N, BN, g.b_ext, g.K, g.two, g.b_part, wid, lane);
  const int all = static_cast<int>((g.K + BK - 1) / BK) << g.two;
  const int k0 = split * g.per_split, k1 = min(all, k0 + g.per_split);
  // Each XCD starts elsewhere in the reduction: rows a power-of-two-like stride
  // apart, all read at the same place at a time, would meet on a few memory
  // channels (65536x7168x256: 254 -> 235 us).
  const int first = k0 + xcd * (k1 - k0) / 8;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));

  // load q of a slice, B's first
  auto load = [&](auto q_tag, const typename OpA::Slice& sa, const typename OpB::Slice& sb,
                  uint32_t at) {
    constexpr int q = decltype(q_tag)::value;
    if constexpr (q < OpB::LOADS) B.load(q, sb, at + OpA::BYTES, wid);
    else A.load(q - OpB::LOADS, sa, at, wid);
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // The K loop on NB of the wavefront's 32-row blocks (block i of the wavefront
  // is block i*WM + wm of the tile, so that a half tile is half of each).
  auto kloop = [&](auto nb_tag) __attribute__((always_inline)) {
    constexpr int NB = decltype(nb_tag)::value;
    constexpr int NP = NB * TN, NF = NB + TN;  // products and fragments of a step
    constexpr int NR = NB * (ACOLS ? 2 : 1) + TN * (BCOLS ? 2 : 1);  // LDS reads of a step
    u32x4 fa[2][NB], fb[2][TN];
    // fragment f of a step, B's first
    auto fragment = [&](int stage, int kk, int to, int f) __attribute__((always_inline)) {
      const char* s = smem + stage * STAGE;
      if (f < TN) fb[to][f] = OpB::fragment(s + OpA::BYTES, kk, wn * (32 * TN) + f * 32, lane);
      else fa[to][f - TN] = OpA::fragment(s, kk, ((f - TN) * WM + wm) * 32, lane);
    };
    auto read = [&](int stage, int kk, int to) __attribute__((always_inline)) {
#pragma unroll
      for (int f = 0; f < NF; ++f) fragment(stage, kk, to, f);
    };
    // B first: each block of acc holds the transposed output block, so four
    // consecutive accumulators are four consecutive columns of one row
    auto product = [&](auto p_tag, int from) __attribute__((always_inline)) {
      constexpr int p = decltype(p_tag)::value;
      acc[p / TN][p % TN] = mma<F16>(fb[from][p % TN], fa[from][p / TN], acc[p / TN][p % TN]);
    };
    // slices in turn from `first` on, around the end
    int ld = first;  // the next slice to load
    auto advance = [&](int k) { return k + 1 == k1 ? k0 : k + 1; };
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int end = s < k1 - k0 ? k1 : 0;
      const auto sa = A.slice(ld, end);
      const auto sb = B.slice(ld, end);
      for_each_index([&](auto q) { load(q, sa, sb, lds0 + s * STAGE); },
                     std::make_integer_sequence<int, NL>{});
      ld = advance(ld);
    }
    wait_vmcnt<(NS - 1) * NL>();
    __syncthreads();
    read(0, 0, 0);
    // A slice: its steps but the last, each reading the next one's fragments
    // behind its own products; then slice kt is read by this wavefront, and the
    // barrier tells that it is by all, and that slice kt+1 has landed; the last
    // step's products then go with the first reads of slice kt+1 and, one after
    // another, the loads of slice kt+NS into the stage that is free.
    static_assert((KK & 1) == 0, "a slice starts with the first fragment set");
    int stage = 0;
    for (int kt = k0; kt < k1; ++kt) {
      const int next = stage + 1 == NS ? 0 : stage + 1;
#pragma unroll
      for (int kk = 0; kk + 1 < KK; ++kk) {
        read(stage, kk + 1, (kk + 1) & 1);
        for_each_index([&](auto p) { product(p, kk & 1); }, std::make_integer_sequence<int, NP>{});
        interleave<NR, NP>();
      }
      const int end = kt + NS < k1 ? k1 : 0;
      const auto sa = A.slice(ld, end);
      const auto sb = B.slice(ld, end);
      ld = advance(ld);
      wait_vmcnt<(NS - 2) * NL>();
      __syncthreads();
      // (pinned: left alone, the scheduler moves the loads behind the products, and
      // every wavefront's loads at once overfill the texture unit's command queue)
      const uint32_t at = lds0 + stage * STAGE;
      constexpr int NQ = NP > NL ? NP : NL;
      for_each_index([&](auto q) {
        constexpr int i = decltype(q)::value;
        if constexpr (i < NP) product(q, 1);
        // the next slice's first fragments behind the first products
        constexpr int PER = (NF + NP - 1) / NP;
#pragma unroll
        for (int f = i * PER; f < (i + 1) * PER && f < NF; ++f) fragment(next, 0, 0, f);
        if constexpr (i < NL) load(q, sa, sb, at);
        __builtin_amdgcn_sched_barrier(0);
      }, std::make_integer_sequence<int, NQ>{});
      stage = next;
    }
  };
  if (TM > 1 && g.M - m0 > (BM / 2) && height == BM) kloop(std::integral_constant<int, TM>{});
  else kloop(std::integral_constant<int, (TM + 1) / 2>{});
  wait_vmcnt<0>();
  __syncthreads();  // the stages are free

  const int64_t m_end = min(g.M, m0 + height);
  // Epilogue, each wavefront by itself: a 32-row block goes to its own LDS
  // part as fp32 (chunks of four columns, swizzled by row) and comes back
  // eight columns of a row to a lane, where rows and columns allow 16-byte
  // accesses, or one column to a lane. A lane keeps its columns for all rows,
  // and a block's residual is fetched while the block before it is finished.
  char* ep = smem + wid * EP;
  constexpr int ECH = 8 * TN;  // 16-byte chunks of a block's row
  auto slot = [](int r, int c) {
    const int key = ECH >= 16 ? (r & 15) : ((r >> 1) & 7);
    return r * (ECH * 16) + ((c ^ key) << 4);
  };
  constexpr int C8 = 4 * TN, RPI = 64 / C8, IT = 32 / RPI;  // rows of one pass of the wavefront
  const int64_t nw = n0 + wn * (32 * TN);                    // the wavefront's first column
  const bool parts = g.splits > 1;
  const bool wide = parts || (g.e.vec && (nw + 32 * TN <= g.N || g.N % 8 == 0));
  const int cols = static_cast<int>(min(int64_t(32 * TN), g.N - nw));  // may be none
  const int c0 = (lane % C8) * 8;  // wide: all eight columns exist, or none
  const int r0 = lane / C8;
  auto block_row = [&](int i) { return m0 + (i * WM + wm) * 32; };
  float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool has_res = wide && !parts && g.e.res;
  u32x4 res[IT];
  auto fetch = [&](int i) __attribute__((always_inline)) {
    const uint16_t* p = g.e.res + block_row(i) * g.e.ldr + nw;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * RPI + r0;
      if (block_row(i) + r < m_end && c0 < cols) res[it] = load8x16(p + (r * int(g.e.ldr) + c0));
    }
  };
  if (wide && !parts && g.e.bias && c0 < cols) {
#pragma unroll
    for (int q = 0; q < 8; ++q) bias[q] = g.e.bias[nw + c0 + q];
  }
  if (has_res) fetch(0);
  for_each_index([&](auto i_tag) {
    constexpr int i = decltype(i_tag)::value;
    const int64_t mb = block_row(i);
    if (mb >= m_end || cols <= 0) return;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(ep + slot(lane & 31, j * 8 + 2 * q + (lane >> 5))) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    // one wavefront's LDS accesses complete in order; the fence keeps the compiler's
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int rows = static_cast<int>(min(int64_t(32), m_end - mb));
    if (wide) {
      u32x4 now[IT];
#pragma unroll
      for (int it = 0; it < IT; ++it) now[it] = res[it];
      if (has_res && i + 1 < TM) fetch(i + 1);
      const Block b(g.e, mb, nw);
      float* part = g.part + (int64_t(split) * g.M + mb) * g.nw + nw;
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int r = it * RPI + r0;
        const f32x4 x = *reinterpret_cast<const f32x4*>(ep + slot(r, 2 * (lane % C8)));
        const f32x4 y = *reinterpret_cast<const f32x4*>(ep + slot(r, 2 * (lane % C8) + 1));
        if (r < rows && c0 < cols) {
          if (parts) {
            float* p = part + (r * int(g.nw) + c0);
            *reinterpret_cast<f32x4*>(p) = x;
            *reinterpret_cast<f32x4*>(p + 4) = y;
          } else {
            float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            finish8(g.e, b, r, c0, v, bias, now[it]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // one pass's values at a time in registers
      }
    } else {
      constexpr int ACROSS = 32 * TN, STEP = 64 / ACROSS, BATCH = 8;
      const int c = lane % ACROSS;
      const Block b(g.e, mb, nw);
      const float b1 = c < cols && g.e.bias ? g.e.bias[nw + c] : 0.f;
#pragma unroll 1
      for (int r = lane / ACROSS; r < 32; r += STEP * BATCH) {
        float z[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
          z[u] = *reinterpret_cast<const float*>(ep + slot(r + u * STEP, c >> 2) + (c & 3) * 4);
        finish_column(g.e, b, r, STEP, c < cols ? rows : 0, c, z, b1);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }, std::make_integer_sequence<int, TM>{});
}

// The sums of the splits, in order, and the epilogue: eight columns a thread (64 threads
// to a workgroup: there are few columns, and they have to spread over the chip).
__global__ __launch_bounds__(64) void linear_join_kernel(GemmArgs g) {
  const int64_t c8 = g.nw / 8;
  const int64_t at = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (at >= g.M * c8) return;
  const int64_t m = at / c8, n = (at - m * c8) * 8;
  const float* p = g.part + m * g.nw + n;
  const int64_t step = g.M * g.nw;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kBatch = 8;  // splits whose loads are in flight together
  for (int s = 0; s < g.splits; s += kBatch) {
    f32x4 x[kBatch], y[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (s + u < g.splits) {
        x[u] = *reinterpret_cast<const f32x4*>(p + (s + u) * step);
        y[u] = *reinterpret_cast<const f32x4*>(p + (s + u) * step + 4);
      }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (s + u < g.splits) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += x[u][i], v[4 + i] += y[u][i];
      }
  }
  const Block b(g.e, m, n);
  if (g.e.vec && n + 8 <= g.N) {
    float bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = g.e.bias ? g.e.bias[n + i] : 0.f;
    finish8(g.e, b, 0, 0, v, bias, b.res ? load8x16(b.res) : u32x4{0, 0, 0, 0});
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float one[1] = {v[i]};
      if (n + i < g.N) finish_column(g.e, b, 0, 1, 1, i, one, g.e.bias ? g.e.bias[n + i] : 0.f);
    }
  }
}

}  // namespace
}  // namespace moe
