// The tile kernel of the 8-bit products (fp8_gemm.hip has the whole picture):
//   c[m, n] = sum over runs b of sa[m, b] sb[n / 128, b] sum over k in run b of a[m, k] w[n, k]
#pragma once

#include "fp8.h"
#include "linear_epilogue.h"
#include "row_tiles.h"
#include "slice_range.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16v8 __attribute__((ext_vector_type(8)));

constexpr int kMaxGroups = 1024;
constexpr int kWaves8 = 8;
constexpr int kThreads8 = 64 * kWaves8;
constexpr uint32_t kPast = 0x80000000u;  // a byte offset past every buffer range
constexpr int kGroupsPer = kMaxGroups / kThreads8;  // groups a thread counts
constexpr int kBandRows = 4;             // row tiles walked together

// kDense    one group of M rows, c through the linear layer's epilogue
// kGrouped  ragged groups, each with a matrix of its own; c as kDense
// kGated    ragged groups with two matrices: h = silu(a w0^T) * (a w1^T), in 8 bits with scales
enum Kind8 { kDense = 0, kGrouped = 1, kGated = 2 };

struct Fp8Args {
  const uint8_t* a;        // [rows, K]
  const float* sa;         // [rows, runs]
  const uint8_t* w0;       // [groups, N, K]
  const uint8_t* w1;       // kGated
  const float* s0;         // [groups, ceil(N / 128), runs]
  const float* s1;
  int K, N, runs;
  int64_t M;               // kDense: rows
  const int32_t* offsets;  // ragged: [groups + 1], counts [groups]
  const int32_t* counts;
  int groups;
  int64_t m_cap;           // no row at or past it is touched
  int max_rows;            // rows of a group past it are not computed
  const int32_t* gather;   // kGated, or nullptr: row r is a[gather[r] / top_k]
  int top_k;
  int64_t tokens;          // gather: rows of a
  int tiles_m, tiles_n, splits, per_split;  // kDense
  float* part;             // splits > 1: [splits, M, nw]
  int64_t nw;
  Epilogue e;              // kDense, kGrouped
  uint8_t* h;              // kGated: [rows, N]
  float* hs;               // [rows, N / 128]
};

// 16 and 4 bytes per lane, memory -> LDS, as dma16, with four more wait states: this kernel has
// places where the compiler restores a scalar operand from a spill right before the
// transfer. They pass while the matrix cores are busy with the product before.
__device__ __forceinline__ void load16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds_addr) {
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc), "s"(soff),
               "{m0}"(lds_addr)
               : "memory");
}
__device__ __forceinline__ void load4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds_addr) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc), "s"(soff),
               "{m0}"(lds_addr)
               : "memory");
}

__device__ __forceinline__ i32x8 join(const u32x4& a, const u32x4& b) {
  return i32x8{int(a[0]), int(a[1]), int(a[2]), int(a[3]), int(b[0]), int(b[1]), int(b[2]), int(b[3])};
}

// Eight e4m3 values as fp16, exactly.
__device__ __forceinline__ f16v8 to_f16(int lo, int hi) {
  const f16v2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
  const f16v2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const f16v2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
  const f16v2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  return f16v8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One run's products of 16 rows of w with 16 rows of a: lane l holds the columns
// 4 (l / 16) .. + 3 (rows of w) of row l % 16. The K order inside the run does not matter,
// as long as both operands have the same.
// The 8-bit instruction adds each 8 neighbouring products after cutting them, towards zero, to multiples
// of 2^-13 of 2^E, E the largest sum of two factors' exponents among them (measured, the 16x16x32 form
// alike; the eights and the runs are added with 24 bits): 1.4e-5 of the result's norm on normal
// values, 3e-6 low on values of one sign, and more where large products cancel. So it is taken where the
// caller asks for it (`fast`) and nowhere else.
__device__ __forceinline__ f32x4 run_product(const i32x8& w, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0,
                                                          0, 0);
}

// The same through fp16, which holds every e4m3 value, at half the rate: sums keep 24 bits
// throughout (1e-8 to 1e-7 of the result's norm).
__device__ __forceinline__ f32x4 run_product_exact(const i32x8& w, const i32x8& a) {
  f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_f16(w[2 * q], w[2 * q + 1]),
                                               to_f16(a[2 * q], a[2 * q + 1]), c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ float silu8(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

// The order of a slice's products: row block by row block, the last two row blocks
// together, so that a w fragment is free for the next slice's as soon as both have read it.
constexpr int block_of(int p, int nb) { return p < (nb - 2) * 4 ? p / 4 : nb - 2 + ((p - (nb - 2) * 4) & 1); }
constexpr int column_of(int p, int nb) { return p < (nb - 2) * 4 ? p % 4 : (p - (nb - 2) * 4) / 2; }

// f(nb) at compile time, for nb from 2 (taken for fewer) to MB, in steps of STEP.
template <int MB, int STEP, class F>
__device__ __forceinline__ void with_blocks(int nb, F&& f) {
  if constexpr (MB - STEP >= 2) {
    if (nb <= MB - STEP) return with_blocks<MB - STEP, STEP>(nb, f);
  }
  f(std::integral_constant<int, MB>{});
}

// The ragged kinds' groups: row tiles before each, rows, first row; sums of the wavefronts.
struct Groups {
  int prefix[kMaxGroups + 1], cnt[kMaxGroups], off[kMaxGroups], wave[2 * kWaves8];
};
struct NoGroups {};

template <int BM, int BN>
constexpr int stage_bytes() {  // rows of a (wave-loads of 64), rows of w, the scales
  return (BM + 63) / 64 * 64 * kRun + BN * kRun + kThreads8 * 4;
}

// The tiles of BM rows x BN staged rows of w, through NS stages.
// WIDE: rows of the outputs go out in 16-byte pieces (always so for the ragged kinds).
// EXACT: products in fp16, sums with 24 bits throughout
template <int BM, int BN, int NS, int KIND, bool WIDE, bool EXACT, class GroupsT>
__device__ __forceinline__ void fp8_tiles(const Fp8Args g, char* const smem, GroupsT& groups, uint32_t* amax_s) {
  constexpr bool GATED = KIND == kGated, RAGGED = KIND != kDense;
  constexpr int WN = BN / 64, WM = kWaves8 / WN, MB = BM / WM / 16;  // a wavefront: 16 MB rows x 64 staged columns
  constexpr int OUT = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int A_BYTES = (BM + 63) / 64 * 64 * kRun, B_BYTES = BN * kRun;
  constexpr int STAGE = stage_bytes<BM, BN>();
  constexpr int AL = (BM + 63) / 64, BL = BN / 64, NL = AL + BL + 1;  // wave-loads of a slice
  constexpr int MS = (MB + 1) / 2 * 2;   // places of a row's scales in a stage
  constexpr int SW = (WM * 16 * MS + 63) / 64;  // the wavefront that brings w's scales; those before it bring the rows'
  static_assert(MB >= 2 && WM * WN == kWaves8 && SW + 1 < kWaves8, "tile");

  const int tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int r15 = lane & 15, grp = lane >> 4;
  const int K = g.K, N = g.N, KT = g.runs;
  const int NT = (N + OUT - 1) / OUT;

  int total;
  if constexpr (RAGGED) {
    // (so many groups over the same rows that their tiles pass kManyTiles compute nothing: sums stop there)
    constexpr int kManyTiles = (1 << 30) - 1;
    int v[kGroupsPer], run = 0;
#pragma unroll
    for (int q = 0; q < kGroupsPer; ++q) {
      const int e = tid * kGroupsPer + q;
      v[q] = e < g.groups ? (groups.cnt[e] + BM - 1) / BM : 0;
      run += v[q];
    }
    int incl = run;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int o = __shfl_up(incl, off, kWave);
      if (lane >= off) incl = min(incl + o, kManyTiles);
    }
    if (lane == kWave - 1) groups.wave[wid] = incl;
    __syncthreads();
    const int before = __shfl_up(incl, 1, kWave);
    int ex = lane > 0 ? before : 0;
    for (int w = 0; w < wid; ++w) ex = min(ex + groups.wave[w], kManyTiles);
#pragma unroll
    for (int q = 0; q < kGroupsPer; ++q) {
      const int e = tid * kGroupsPer + q;
      if (e < g.groups) groups.prefix[e] = ex;
      ex = min(ex + v[q], kManyTiles);
    }
    if (tid == kThreads8 - 1) groups.prefix[g.groups] = ex;
    __syncthreads();
    const int64_t all = int64_t(uniform(groups.prefix[g.groups])) * NT;
    total = all < kManyTiles ? int(all) : 0;
  } else {
    total = g.tiles_m * NT * g.splits;
  }

  const int G = gridDim.x;
  int slot = blockIdx.x;
  if ((G & 7) == 0) slot = (blockIdx.x & 7) * (G >> 3) + (blockIdx.x >> 3);

  struct Tile {
    int64_t row0;  // first row of a (without a gather) and of the outputs
    int rows, n0, e, split;
  };
  // Tile ids run group by group, inside a group in bands of kBandRows row tiles, column tile
  // major inside a band: the 32 neighbours of an XCD share the rows of 4 row tiles
  // and the columns of 8 column tiles behind one L2.
  auto locate = [&](int id) __attribute__((always_inline)) {
    Tile t;
    int mtiles, rem, rows;
    if constexpr (RAGGED) {
      int lo = 0, hi = g.groups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (groups.prefix[mid] * NT <= id) lo = mid; else hi = mid - 1;
      }
      t.e = uniform(lo);
      t.split = 0;
      mtiles = uniform(groups.prefix[t.e + 1] - groups.prefix[t.e]);
      rem = id - uniform(groups.prefix[t.e]) * NT;
      rows = uniform(groups.cnt[t.e]);
    } else {
      const int tiles = g.tiles_m * NT;
      t.e = 0;
      t.split = id / tiles;
      mtiles = g.tiles_m;
      rem = id - t.split * tiles;
      rows = 0;
    }
    const int full = mtiles / kBandRows * kBandRows;
    int nt, mt;
    if (rem < full * NT) {
      const int band = rem / (kBandRows * NT), r2 = rem % (kBandRows * NT);
      nt = r2 / kBandRows;
      mt = band * kBandRows + r2 % kBandRows;
    } else {
      const int tail = mtiles - full, r2 = rem - full * NT;
      nt = r2 / tail;
      mt = full + r2 % tail;
    }
    t.n0 = nt * OUT;
    if constexpr (RAGGED) {
      // a group's 16-row blocks dealt out evenly: no short last tile
      const int blks = (rows + 15) / 16, bq = blks / mtiles, br = blks % mtiles;
      const int start = 16 * (mt * bq + min(mt, br));
      t.rows = min((bq + (mt < br ? 1 : 0)) * 16, rows - start);
      t.row0 = int64_t(uniform(groups.off[t.e])) + start;
    } else {
      t.row0 = int64_t(mt) * BM;
      t.rows = uniform(int(min(int64_t(BM), g.M - t.row0)));
    }
    return t;
  };

  // ---- operands of the current tile
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
  // This lane's place in a wave-load of 8 rows x 128 bytes: row lane / 8, physical
  // chunk lane % 8. The 16 rows that an LDS cycle reads at one logical chunk have to lie in
  // 16 different bank groups; a row's parity picks a half of the banks, its key the
  // chunk. a is read in runs of 16 rows, w in the rows 8 i + j and 8 i + 4 + j, i, j < 4.
  const int ld_r = wid * 8 + lane / 8;
  const int a_ch = (lane & 7) ^ ((ld_r >> 1) & 7);
  const int b_ch = (lane & 7) ^ (((ld_r >> 1) & 1) | (((ld_r >> 3) & 3) << 1));
  uint32_t oa[AL], ob[BL], osc;
  i32x4 ra, rb0, rb1, rsc;

  auto setup = [&](const Tile& t) __attribute__((always_inline)) {
    const int64_t wrow = int64_t(t.e) * N + t.n0;
    const int valid = min(OUT, N - t.n0);
    const bool gathered = GATED && g.gather;
    const int64_t a0 = gathered ? 0 : t.row0;
    const uint32_t a_rows = gathered ? uint32_t(g.tokens) : uint32_t(t.rows);
    // a row of the tile as a row of the range, or -1
    auto source = [&](int r) {
      if (r >= t.rows) return -1;
      if (!gathered) return r;
      const int src = g.gather[t.row0 + r];
      const int token = src / g.top_k;
      return src >= 0 && token < g.tokens ? token : -1;
    };
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int r = source(ld_r + 64 * i);
      oa[i] = r >= 0 ? uint32_t(r) * uint32_t(K) + uint32_t(a_ch) * 16u : kPast;
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int r = (ld_r + 64 * i) % OUT;
      ob[i] = r < valid ? uint32_t(r) * uint32_t(K) + uint32_t(b_ch) * 16u : kPast;
    }
    ra = make_rsrc(g.a + a0 * K, a_rows * uint32_t(K));
    rb0 = make_rsrc(g.w0 + wrow * K, uint32_t(valid) * uint32_t(K));
    rb1 = GATED ? make_rsrc(g.w1 + wrow * K, uint32_t(valid) * uint32_t(K)) : rb0;
    // scales: wavefronts before SW bring the rows', each wavefront row's MB blocks next to
    // each other; SW those of w (two runs of columns, or w0's) and, gated, SW + 1 those of w1
    osc = kPast;
    if (wid < SW) {
      const int s = wid * 64 + lane, w = s / MS;
      const int r = s % MS < MB ? source(((s % MS) * WM + w / 16) * 16 + (w & 15)) : -1;
      if (r >= 0) osc = uint32_t(r) * uint32_t(KT) * 4u;
      rsc = make_rsrc(g.sa + a0 * KT, a_rows * uint32_t(KT) * 4u);
    } else {
      const int nblocks = (N + kRun - 1) / kRun;
      const int left = min(GATED ? 1 : 2, nblocks - t.n0 / kRun);
      const float* s = (GATED && wid > SW ? g.s1 : g.s0) + (int64_t(t.e) * nblocks + t.n0 / kRun) * KT;
      rsc = make_rsrc(s, uint32_t(left) * uint32_t(KT) * 4u);
      if (lane < left && wid <= SW + (GATED ? 1 : 0)) osc = uint32_t(lane) * uint32_t(KT) * 4u;
    }
  };
  // Wave-load q of a slice, by these resources and lane offsets, into the stage at `at`.
  struct Sources {
    i32x4 a, b0, b1, s;
    uint32_t slice;
  };
  auto load = [&](auto q_tag, const Sources& from, uint32_t at, const uint32_t (&va)[AL],
                  const uint32_t (&vb)[BL], uint32_t vs) __attribute__((always_inline)) {
    constexpr int q = decltype(q_tag)::value;
    if constexpr (q < BL)
      load16(GATED && q >= BL / 2 ? from.b1 : from.b0, vb[q], from.slice * kRun,
             at + A_BYTES + (wid + kWaves8 * q) * 1024);
    else if constexpr (q < BL + AL)
      load16(from.a, va[q - BL], from.slice * kRun, at + (wid + kWaves8 * (q - BL)) * 1024);
    else if constexpr (q < NL)
      load4(from.s, vs, from.slice * 4u, at + A_BYTES + B_BYTES + wid * 256);
  };
  // A slice at or past `end` reads nothing but zeros, by an empty range without an offset. (Scalar
  // work: more than about five vector instructions to a product no longer fit beside it.)
  auto upto = [&](int kt, int end) __attribute__((always_inline)) {
    Sources f{ra, rb0, rb1, rsc, slice_range(kt, end, 0).slice};
    auto bytes = [&](const i32x4& r) { return int(slice_range(kt, end, uint32_t(r[2])).bytes); };
    f.a[2] = bytes(ra), f.b0[2] = bytes(rb0), f.b1[2] = bytes(rb1), f.s[2] = bytes(rsc);
    return f;
  };
  // The first slices of a range, all stages; a chunk past K reads zeros too.
  auto first_slices = [&](int k0, int k1) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int left = K - (k0 + s) * kRun;
      uint32_t va[AL], vb[BL];
#pragma unroll
      for (int i = 0; i < AL; ++i) va[i] = a_ch * 16 < left ? oa[i] : kPast;
#pragma unroll
      for (int i = 0; i < BL; ++i) vb[i] = b_ch * 16 < left ? ob[i] : kPast;
      const Sources f = upto(k0 + s, k1);
      for_each_index([&](auto q) { load(q, f, lds0 + s * STAGE, va, vb, osc); },
                     std::make_integer_sequence<int, NL>{});
    }
  };

  f32x4 acc[MB][4];

  // Where this lane reads in the stage at hand: a's fragments (two halves; block i of the
  // wavefront is block i WM + wm of the tile, so that a partly filled tile is shared out
  // evenly), w's, and the scales.
  struct Place {
    int a, a2, b, b2, s, w;
  };
  auto place = [&]() {
    Place x;
    x.a = (wm * 16 + r15) * kRun + ((grp ^ (r15 >> 1)) << 4);
    x.b = A_BYTES + (wn * (GATED ? 32 : 64) + 8 * (r15 >> 2) + (r15 & 3)) * kRun +
          ((grp ^ (((r15 >> 1) & 1) | ((r15 >> 2) << 1))) << 4);
    x.a2 = x.a ^ 64, x.b2 = x.b ^ 64;
    x.s = A_BYTES + B_BYTES + (wm * 16 + r15) * (MS * 4);
    x.w = A_BYTES + B_BYTES + SW * 256 + (GATED ? 0 : wn * 64 / kRun * 4);
    asm volatile("" : "+v"(x.a), "+v"(x.b), "+v"(x.a2), "+v"(x.b2), "+v"(x.s), "+v"(x.w));
    return x;
  };
  auto move = [&](Place& x, int by) __attribute__((always_inline)) {
    x.a += by, x.a2 += by, x.b += by, x.b2 += by, x.s += by, x.w += by;
  };
  auto read_a = [&](const Place& x, int i) __attribute__((always_inline)) {
    const int o = i * WM * (16 * kRun);
    return join(*reinterpret_cast<const u32x4*>(smem + x.a + o),
                *reinterpret_cast<const u32x4*>(smem + x.a2 + o));
  };
  auto read_b = [&](const Place& x, int j) __attribute__((always_inline)) {
    const int o = ((j >> 1) * (GATED ? OUT : 32) + 4 * (j & 1)) * kRun;
    return join(*reinterpret_cast<const u32x4*>(smem + x.b + o),
                *reinterpret_cast<const u32x4*>(smem + x.b2 + o));
  };
  // block i's row scale goes to sa[i % 4], two blocks' at a time
  auto read_sa = [&](const Place& x, int pair, float (&sa)[4]) __attribute__((always_inline)) {
    const f32x2 v = *reinterpret_cast<const f32x2*>(smem + x.s + pair * 8);
    sa[2 * (pair & 1)] = v[0], sa[2 * (pair & 1) + 1] = v[1];
  };
  auto read_sw = [&](const Place& x, float (&sb)[2]) __attribute__((always_inline)) {
    sb[0] = *reinterpret_cast<const float*>(smem + x.w);
    sb[1] = GATED ? *reinterpret_cast<const float*>(smem + x.w + 256) : sb[0];
  };
  // Waits for a range's first slice. Of the tile before, `stores` stores at least were issued
  // behind the slices' loads; loads and stores complete in order, so those may be outstanding too.
  int stores = 0;
  auto wait_first = [&]() __attribute__((always_inline)) {
    if (stores >= 16) wait_vmcnt<(NS - 1) * NL + 16>();
    else if (stores >= 8) wait_vmcnt<(NS - 1) * NL + 8>();
    else wait_vmcnt<(NS - 1) * NL>();
  };
  auto scaled_add = [&](f32x4& to, const f32x4& p, float s) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) to[q] = __builtin_fmaf(p[q], s, to[q]);
  };

  // The K loop on NB of the wavefront's row blocks.
  auto kloop = [&](auto nb_tag, int k0, int k1) __attribute__((always_inline)) {
    constexpr int NB = decltype(nb_tag)::value, NP = NB * 4, LAST = (NB - 2) * 4;
    i32x8 fa[3], fb[4];  // block i's a fragment is in fa[(i + phase) % 3]
    f32x4 part[4];
    float sa[4], sb[2], s_old[2];
    Place x = place();
    wait_first();
    __syncthreads();
    read_sw(x, sb);
    read_sa(x, 0, sa);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < 2) fa[j] = read_a(x, j);
      fb[j] = read_b(x, j);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) part[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    s_old[0] = s_old[1] = 0.f;
    int stage = 0;
    // One slice: each step is a product and the scaled addition of the product three
    // steps before. All of the slice is read when the last two row blocks' products
    // begin: the barrier there tells that it is by every wavefront and that the next
    // slice has landed; the loads into the free stage and the reads of the next slice's
    // first fragments go between those products, one each, or every
    // wavefront's at once would fill the queues and hold up the products.
    // EARLY: when the third row block begins, w's part of the stage and the rows of the first four
    // blocks are read already: a barrier there lets EL of the loads go ahead, which then
    // have one and a half slices to land instead of one.
    constexpr bool EARLY = WM == 2 && NB >= 5;
    constexpr int EL = !EARLY ? 0 : BL + 2 < LAST - 8 ? BL + 2 : LAST - 8;
    auto slice = [&](int kt, auto phase_tag) __attribute__((always_inline)) {
      constexpr int PH = decltype(phase_tag)::value, PN = (PH + NB) % 3;
      const uint32_t at = lds0 + stage * STAGE;
      const Sources from = upto(kt + NS, k1);
      auto load_next = [&](auto q) __attribute__((always_inline)) { load(q, from, at, oa, ob, osc); };
      for_each_index([&](auto p_tag) __attribute__((always_inline)) {
        constexpr int p = decltype(p_tag)::value, i = block_of(p, NB), j = column_of(p, NB);
        if constexpr (EARLY && p == 8) __syncthreads();
        if constexpr (p == LAST) {
          wait_vmcnt<(NS - 2) * NL + EL>();
          __syncthreads();
          // from here on the next stage is read
          const bool wrap = stage + 1 == NS;
          move(x, wrap ? -(NS - 1) * STAGE : STAGE);
          stage = wrap ? 0 : stage + 1;
        }
        if constexpr (EARLY && p >= 8 && p < 8 + EL)
          load_next(std::integral_constant<int, p - 8>{});
        // the product three steps back, of this slice or the last one
        constexpr int o = p >= 3 ? p - 3 : NP - 3 + p;
        constexpr int oi = block_of(o, NB), oj = column_of(o, NB);
        const f32x4 old = part[o & 3];
        float s;
        if constexpr (p >= 3) s = sa[oi & 3] * sb[oj >> 1];
        else s = s_old[oi - (NB - 2)];
        part[p & 3] = run_product(fb[j], fa[(i + PH) % 3]);
        scaled_add(acc[oi][oj], old, s);
        if constexpr (p < LAST) {
          if constexpr (j == 0 && i + 2 < NB) fa[(i + 2 + PH) % 3] = read_a(x, i + 2);
          if constexpr (j == 3 && i % 2 == 0 && i + 2 < NB) read_sa(x, i / 2 + 1, sa);
        } else {
          constexpr int q = p - LAST;
          load_next(std::integral_constant<int, EL + q>{});
          if constexpr (q == 7 && EL + 8 < NL) load_next(std::integral_constant<int, EL + 8>{});
          static_assert(NL <= 9, "loads fit the steps behind the barrier");
          if constexpr (q == 0) fa[PN] = read_a(x, 0);
          if constexpr (q == 7) fa[(1 + PN) % 3] = read_a(x, 1);
          if constexpr (q & 1) fb[q / 2] = read_b(x, q / 2);
        }
        __builtin_amdgcn_sched_barrier(0);
      }, std::make_integer_sequence<int, NP>{});
      // the last three products are of columns 2 (block NB - 1) and 3
      s_old[0] = sa[(NB - 2) & 3] * sb[1];
      s_old[1] = sa[(NB - 1) & 3] * sb[1];
      read_sw(x, sb);
      read_sa(x, 0, sa);
    };
    int kt = k0;
    if constexpr (NB % 3 == 0) {
      for (; kt < k1; ++kt) slice(kt, std::integral_constant<int, 0>{});
    } else {
      for (; kt + 2 < k1; kt += 3) {
        slice(kt, std::integral_constant<int, 0>{});
        slice(kt + 1, std::integral_constant<int, NB % 3>{});
        slice(kt + 2, std::integral_constant<int, 2 * NB % 3>{});
      }
      if (kt < k1) slice(kt++, std::integral_constant<int, 0>{});
      if (kt < k1) slice(kt, std::integral_constant<int, NB % 3>{});
    }
#pragma unroll
    for (int p = NP - 3; p < NP; ++p)
      scaled_add(acc[block_of(p, NB)][column_of(p, NB)], part[p & 3], s_old[block_of(p, NB) - (NB - 2)]);
  };

  // The same with the products in fp16. A step is two columns' products of a block, their
  // instructions in turn (each column's are a chain), with the vector work between them:
  // the scaled addition of the step before, and the conversion of fragments
  // that come up, half of the next row block's each step; w's for the next slice, two
  // columns' each, in the last step of a slice and the first one of the next.
  auto kloop_exact = [&](auto nb_tag, int k0, int k1) __attribute__((always_inline)) {
    constexpr int NB = decltype(nb_tag)::value;
    f16v8 bh[4][4], ah[2][4];  // block i's a fragment is in ah[(i + phase) % 2], as is a8's
    i32x8 a8[2], b8[2];
    f32x4 part[2][2];
    float sa[4], sb[2], s_old = 0.f;
    Place x = place();
    auto convert = [&](f16v8& to, const i32x8& from, int q) __attribute__((always_inline)) {
      to = to_f16(from[2 * q], from[2 * q + 1]);
    };
    wait_first();
    __syncthreads();
    read_sw(x, sb);
    read_sa(x, 0, sa);
    a8[0] = read_a(x, 0), a8[1] = read_a(x, 1);
    b8[0] = read_b(x, 0), b8[1] = read_b(x, 1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      convert(ah[0][q], a8[0], q);
      convert(bh[0][q], b8[0], q);
      convert(bh[1][q], b8[1], q);
      bh[2][q] = bh[3][q] = bh[0][q];
    }
    b8[0] = read_b(x, 2), b8[1] = read_b(x, 3);
#pragma unroll
    for (int q = 0; q < 4; ++q) part[q >> 1][q & 1] = f32x4{0.f, 0.f, 0.f, 0.f};
    int stage = 0;
    auto slice = [&](int kt, auto phase_tag) __attribute__((always_inline)) {
      constexpr int PH = decltype(phase_tag)::value;
      const uint32_t at = lds0 + stage * STAGE;
      const Sources from = upto(kt + NS, k1);
      auto load_next = [&](auto q) __attribute__((always_inline)) { load(q, from, at, oa, ob, osc); };
      for_each_index([&](auto t_tag) __attribute__((always_inline)) {
        constexpr int t = decltype(t_tag)::value, i = t >> 1, h = t & 1;
        constexpr bool first = t == 0, last = t == 2 * NB - 1;
        if constexpr (t == 2 * NB - 4) {
          // this slice is read, the next one has landed
          wait_vmcnt<(NS - 2) * NL>();
          __syncthreads();
          const bool wrap = stage + 1 == NS;
          move(x, wrap ? -(NS - 1) * STAGE : STAGE);
          stage = wrap ? 0 : stage + 1;
        }
        if constexpr (h == 0) a8[(i + PH) & 1] = read_a(x, i + 2 < NB ? i + 2 : i + 2 - NB);
        if constexpr (h == 1 && i % 2 == 0 && i + 2 < NB) read_sa(x, i / 2 + 1, sa);
        if constexpr (t == 2 * NB - 3) b8[0] = read_b(x, 0), b8[1] = read_b(x, 1);
        if constexpr (t >= 2 * NB - 4) {
          constexpr int z = t - (2 * NB - 4);
          load_next(std::integral_constant<int, 2 * z>{});
          load_next(std::integral_constant<int, 2 * z + 1>{});
          if constexpr (z == 3) load_next(std::integral_constant<int, 8>{});
        }
        // the step before: column pair 1 - h
        constexpr int oi = first ? NB - 1 : (t - 1) >> 1, oh = 1 - h;
        const f32x4 old0 = part[oh][0], old1 = part[oh][1];
        float s;
        if constexpr (first) s = s_old;
        else s = sa[oi & 3] * sb[oh];
        f32x4 c0{0.f, 0.f, 0.f, 0.f}, c1 = c0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          c0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(bh[2 * h][q], ah[(i + PH) & 1][q], c0, 0, 0, 0);
          c1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(bh[2 * h + 1][q], ah[(i + PH) & 1][q], c1, 0, 0, 0);
        }
        part[h][0] = c0, part[h][1] = c1;
        scaled_add(acc[oi][2 * oh], old0, s);
        scaled_add(acc[oi][2 * oh + 1], old1, s);
#pragma unroll
        for (int q = 2 * h; q < 2 * h + 2; ++q) convert(ah[(i + 1 + PH) & 1][q], a8[(i + 1 + PH) & 1], q);
        if constexpr (first || last) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            convert(bh[first ? 2 : 0][q], b8[0], q);
            convert(bh[first ? 3 : 1][q], b8[1], q);
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                        // a product
          __builtin_amdgcn_sched_group_barrier(0x002, first || last ? 7 : 3, 0);    // vector work
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (last) b8[0] = read_b(x, 2), b8[1] = read_b(x, 3);
      }, std::make_integer_sequence<int, 2 * NB>{});
      s_old = sa[(NB - 1) & 3] * sb[1];
      read_sw(x, sb);
      read_sa(x, 0, sa);
    };
    int kt = k0;
    if constexpr (NB % 2 == 0) {
      for (; kt < k1; ++kt) slice(kt, std::integral_constant<int, 0>{});
    } else {
      for (; kt + 1 < k1; kt += 2) {
        slice(kt, std::integral_constant<int, 0>{});
        slice(kt + 1, std::integral_constant<int, 1>{});
      }
      if (kt < k1) slice(kt, std::integral_constant<int, 0>{});
    }
    scaled_add(acc[NB - 1][2], part[1][0], s_old);
    scaled_add(acc[NB - 1][3], part[1][1], s_old);
  };

  // ---- outputs
  auto column_bias = [&](int64_t n, float (&bias)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) bias[q] = g.e.bias && n < N ? g.e.bias[n + q] : 0.f;
  };
  // A row's scale from its wavefronts' largest magnitudes, and its e4m3 values.
  auto amax_row = [&](uint32_t m) {
    m = max(m, uint32_t(__shfl_xor(int(m), 16, kWave)));
    return max(m, uint32_t(__shfl_xor(int(m), 32, kWave)));
  };

  auto epilogue = [&](const Tile& t) __attribute__((always_inline)) {
    // (hidden from the compiler, which would keep every block's addresses, all tiles long)
    int r15 = lane & 15, grp = lane >> 4;
    asm volatile("" : "+v"(r15), "+v"(grp));
    if constexpr (GATED) {
      float hv[MB][8];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if ((i * WM + wm) * 16 >= t.rows) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) hv[i][q] = silu8(acc[i][q >> 2][q & 3]) * acc[i][2 + (q >> 2)][q & 3];
        const uint32_t m = amax_row(magnitude(hv[i]));
        if (grp == 0) amax_s[wn * BM + (i * WM + wm) * 16 + r15] = m;
        __builtin_amdgcn_sched_barrier(0);  // one block's values at a time in registers
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int r = (i * WM + wm) * 16 + r15;
        if (r >= t.rows) continue;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < WN; ++w) m = max(m, amax_s[w * BM + r]);
        const float s = scale_of(m);
        const int64_t row = t.row0 + r;
        store_fp8x8(g.h, row * N + t.n0 + wn * 32 + grp * 8, to_fp8x8(hv[i], 1.f / s));
        if (wn == 0 && grp == 0) g.hs[row * (N / kRun) + t.n0 / kRun] = s;
        __builtin_amdgcn_sched_barrier(0);
      }
    } else if constexpr (WIDE) {
      const bool parts = KIND == kDense && g.splits > 1;
      const int64_t nw = t.n0 + wn * 64;
      // Nothing to do but to add a residual, to round and to store: without the general form's
      // vector work, which took a third of a tile's time at six runs (65536x768x2048, fast: 157 -> 133 us, now 128).
      // Two neighbouring lanes' rows change halves, so that a store, and a load of the residual, takes
      // 128 bytes of a row and not 64: first the even rows, then the odd ones (65536x2048x7168, fast: 961 -> 910 us,
      // with a residual 1152 -> 1085).
      auto store_rows = [&](auto res_tag) __attribute__((always_inline)) {
        constexpr bool RES = decltype(res_tag)::value;
        const bool odd = r15 & 1;
        const int64_t row = t.row0 + wm * 16 + (r15 & ~1), col = nw + 32 * (r15 & 1) + 8 * grp;
        const bool in = col < N;
        uint16_t* o = static_cast<uint16_t*>(g.e.out) + row * g.e.ldo + col;
        const uint16_t* p = RES ? g.e.res + row * g.e.ldr + col : nullptr;
        // (x, y): columns 0-31 and 32-63 of the lane's row <-> its part of the even and of the odd row
        auto trade = [&](u32x4& x, u32x4& y) __attribute__((always_inline)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t a = x[q], b = y[q], got = dpp<0xb1>(odd ? a : b);
            x[q] = odd ? got : a, y[q] = odd ? b : got;
          }
        };
        u32x4 res[2];
        auto fetch = [&](int i) __attribute__((always_inline)) {
          const int r = (i * WM + wm) * 16 + (r15 & ~1);
          if (in && r < t.rows) res[0] = load8x16(p);
          if (in && r + 1 < t.rows) res[1] = load8x16(p + g.e.ldr);
          p += WM * 16 * g.e.ldr;
        };
        if constexpr (RES) fetch(0);
#pragma unroll
        for (int i = 0; i < MB; ++i, o += WM * 16 * g.e.ldo) {
          u32x4 now[2] = {res[0], res[1]};
          if (RES && i + 1 < MB) fetch(i + 1);
          if ((i * WM + wm) * 16 >= t.rows) continue;
          if constexpr (RES) trade(now[0], now[1]);
          u32x4 out[2];
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = acc[i][2 * jj + (q >> 2)][q & 3];
            if constexpr (RES) {
              float x[8];
              unpack8x16(now[jj], x, g.e.f16);
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] += x[q];
            }
            out[jj] = KIND == kGrouped ? pack8(v) : pack8x16(v, g.e.f16);
          }
          trade(out[0], out[1]);
          const int r = (i * WM + wm) * 16 + (r15 & ~1);
          if (in && r < t.rows) __builtin_nontemporal_store(out[0], reinterpret_cast<u32x4*>(o));
          if (in && r + 1 < t.rows) __builtin_nontemporal_store(out[1], reinterpret_cast<u32x4*>(o + g.e.ldo));
          if constexpr (RES) __builtin_amdgcn_sched_barrier(0);
        }
      };
      if constexpr (KIND == kGrouped) return store_rows(std::false_type{});
      if (!parts && !g.e.bias && g.e.act == MOE_ACT_NONE && !g.e.out_f32)
        return g.e.res ? store_rows(std::true_type{}) : store_rows(std::false_type{});
      float bias[2][8];
      if (!parts) {
        column_bias(nw + grp * 8, bias[0]);
        column_bias(nw + 32 + grp * 8, bias[1]);
      }
      const Block b(g.e, t.row0, nw);
      // the residual, a block ahead of its use
      const bool has_res = KIND == kDense && !parts && g.e.res;
      u32x4 res[2];
      auto fetch = [&](int i) __attribute__((always_inline)) {
        const int r = (i * WM + wm) * 16 + r15;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int c = 32 * jj + 8 * grp;
          if (r < t.rows && nw + c < N) res[jj] = load8x16(b.res + (r * b.ldr + c));
        }
      };
      if (has_res) fetch(0);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int r = (i * WM + wm) * 16 + r15;
        if ((i * WM + wm) * 16 >= t.rows) continue;
        const u32x4 now[2] = {res[0], res[1]};
        if (has_res && i + 1 < MB) fetch(i + 1);
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int c = 32 * jj + 8 * grp;
          if (r >= t.rows || nw + c >= N) continue;
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = acc[i][2 * jj + (q >> 2)][q & 3];
          if (parts) {
            float* p = g.part + (int64_t(t.split) * g.M + t.row0 + r) * g.nw + nw + c;
            *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
          } else {
            finish8(g.e, b, r, c, v, bias[jj], now[jj]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // one block's values at a time in registers
      }
    } else {
      // rows of any alignment: a block of 16 rows x 64 columns through LDS, then a column to a lane
      constexpr int ROW = 68;  // floats of an LDS row: rows 4 banks apart
      float* ep = reinterpret_cast<float*>(smem) + wid * (16 * ROW);
      const int64_t nw = t.n0 + wn * 64;
      const int cols = int(min(int64_t(64), N - nw));
      const float b1 = lane < cols && g.e.bias ? g.e.bias[nw + lane] : 0.f;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int rb = (i * WM + wm) * 16;
        if (rb >= t.rows || cols <= 0) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4*>(ep + r15 * ROW + 32 * (j >> 1) + 8 * grp + 4 * (j & 1)) = acc[i][j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const Block b(g.e, t.row0 + rb, nw);
#pragma unroll 1
        for (int r = 0; r < 16; r += 8) {
          float z[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) z[u] = ep[(r + u) * ROW + lane];
          finish_column(g.e, b, r, 1, lane < cols ? min(16, t.rows - rb) : 0, lane, z, b1);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
    }
  };

  // ---- the tiles
  // A tile's reduction: its whole runs, and by itself a last one that K does not fill.
  const int whole = K / kRun;
  auto segment = [&](const Tile& t, int& k0, int& k1, int& end) __attribute__((always_inline)) {
    k0 = KIND == kDense ? t.split * g.per_split : 0;
    end = KIND == kDense ? min(KT, k0 + g.per_split) : KT;
    k1 = KIND == kDense && k0 < whole ? min(end, whole) : end;
  };
  auto begin = [&](const Tile& t) __attribute__((always_inline)) {
    int k0, k1, end;
    segment(t, k0, k1, end);
    setup(t);
    first_slices(k0, k1);
  };
  int id = slot;
  if (id >= total) return;
  Tile t = locate(id);
  begin(t);
  for (;;) {
    int k0, k1, end;
    segment(t, k0, k1, end);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nb = ((t.rows + 15) / 16 + WM - 1) / WM;  // row blocks of a wavefront
    auto reduce = [&](auto b, int from, int to) __attribute__((always_inline)) {
      if constexpr (EXACT) kloop_exact(b, from, to);
      else kloop(b, from, to);
      wait_vmcnt<0>();
      __syncthreads();  // the stages are free
    };
    with_blocks<MB, RAGGED ? 1 : 2>(nb, [&](auto b) __attribute__((always_inline)) { reduce(b, k0, k1); });
    if constexpr (!RAGGED) {
      if (k1 < end) {
        stores = 0;
        first_slices(k1, end);
        reduce(std::integral_constant<int, MB>{}, k1, end);
      }
    }
    id += G;
    if (id >= total) {
      epilogue(t);
      return;
    }
    const Tile now = t;
    t = locate(id);
    if constexpr (WIDE) {
      begin(t);  // the next tile's first slices are on their way during this one's epilogue
      epilogue(now);
      // each row block with rows in it stores once, or twice where the columns are all there and it
      // has more than one row
      const int blocks = now.rows > wm * 16 ? (now.rows - wm * 16 + 16 * WM - 1) / (16 * WM) : 0;
      stores = GATED ? blocks : now.n0 + wn * 64 + 64 <= N ? 2 * blocks - (now.rows % 16 == 1) : 0;
    } else {
      epilogue(now);
      __syncthreads();  // LDS is read out before it is written again
      begin(t);
    }
  }
}

// FEW > 0: row tiles of FEW rows with a third stage, where the groups are so small that this makes
// few more tiles: less of a stage is rows that are not there, and more of w is on its way. 32 groups,
// 7168 and 2048 wide, full-width sums, gate/up and down with 160 rows a tile against 64: groups of 32 rows
// 196 -> 167 us and 117 -> 104, of 128 (twice the tiles) 234 -> 294 and 139 -> 155, of 256 436 -> 525 and
// 232 -> 288; skewed groups' gate/up with 1.22 times the tiles 223 -> 208, with 1.47 times 204 -> 227. fast,
// 256 rows against 64: groups of 32 203 -> 162 and 114 -> 98, of 100 (twice) 215 -> 225 and 122 -> 119, of
// 160 (three times) 214 -> 311 and 122 -> 172. So up to 5/4 times the tiles, and fast's down up to twice.
// (Where the large tile is taken it is as fast as in a kernel without the small one: groups of 256 to 2048 rows
// and skewed ones within 2 %, fast's gate/up 2 to 7 % faster.)
template <int BM, int BN, int NS, int KIND, bool WIDE, bool EXACT, int FEW>
__global__ __launch_bounds__(kThreads8, 1) void fp8_kernel(Fp8Args g) {
  constexpr bool RAGGED = KIND != kDense;
  constexpr int LDS = NS * stage_bytes<BM, BN>(), LDS_FEW = FEW ? 3 * stage_bytes<FEW ? FEW : BM, BN>() : 0;
  __shared__ __attribute__((aligned(1024))) char smem[LDS > LDS_FEW ? LDS : LDS_FEW];
  __shared__ std::conditional_t<RAGGED, Groups, NoGroups> groups;
  __shared__ uint32_t amax_s[KIND == kGated ? BN / 64 * BM : 1];
  if constexpr (RAGGED) {
    // a group's rows stay inside [0, m_cap) whatever the device's counts say
    const int tid = threadIdx.x;
    int tiles = 0, few = 0;
#pragma unroll
    for (int q = 0; q < kGroupsPer; ++q) {
      const int e = tid * kGroupsPer + q;
      if (e >= g.groups) continue;
      const int o = g.offsets[e];
      const int64_t room = o < 0 ? 0 : max(int64_t(0), g.m_cap - o);
      const int c = int(min(int64_t(min(max(g.counts[e], 0), g.max_rows)), room));
      groups.cnt[e] = c, groups.off[e] = o;
      if constexpr (FEW > 0) tiles += choice_tiles(c, BM), few += choice_tiles(c, FEW);
    }
    if constexpr (FEW > 0) {
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1)
        tiles += __shfl_xor(tiles, off, kWave), few += __shfl_xor(few, off, kWave);
      const int wid = tid / kWave;
      if (lane_id() == 0) groups.wave[wid] = tiles, groups.wave[kWaves8 + wid] = few;
      __syncthreads();
      tiles = few = 0;
#pragma unroll
      for (int w = 0; w < kWaves8; ++w) tiles += groups.wave[w], few += groups.wave[kWaves8 + w];
      __syncthreads();
      if (takes_small(uniform(few), uniform(tiles), KIND == kGated || EXACT ? 5 : 8))
        return fp8_tiles<FEW, BN, 3, KIND, WIDE, EXACT>(g, smem, groups, amax_s);
    }
  }
  fp8_tiles<BM, BN, NS, KIND, WIDE, EXACT>(g, smem, groups, amax_s);
}

// The sums of the splits, in order, and the epilogue: eight columns a thread.
__global__ __launch_bounds__(64) void fp8_join_kernel(Fp8Args g) {
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
