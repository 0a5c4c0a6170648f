// Routing by softmax or sigmoid scores with a selection bias and expert groups,
// and the gradient of its weights.
//
//   s_e = sigmoid(l_e)  or  softmax(l)_e over all E experts
//   v_e = s_e + bias_e                                  (v = s without a bias)
//   a group's rank is its largest v, or the sum of its two largest
//   of the top_groups best groups, the k experts with the largest v
//   w_j = scale * s_j, or scale * s_j / sum over the k selected
//
// ties to the lower index throughout.
//
// The choice is that of fp64 scores: an fp32 sigmoid rounds by up to 2^-24, and
// at 65536 tokens of 256 experts a few tokens have two candidates closer than
// that. fp64 exponentials for every expert are what the first form of this
// kernel spent its time on (87 us for those 65536 tokens), so the scores are
// formed in fp32 with a bound on their error, and the choice stands where
// neighbouring candidates lie further apart than the bound allows (or are
// equal in logit and bias, a true tie). Where they do not, about one wavefront
// in a hundred, fp64 values order the candidates or, where the candidates
// themselves are in doubt, the wavefront chooses again from fp64 scores.
//
// G lanes (8 to 64, inside one wavefront) own a token. A lane's experts all
// belong to one group: lpg (a power of two) consecutive lanes hold a group,
// cpl consecutive experts each, so a group's rank is a butterfly over lpg lanes.
#include <cfloat>
#include <climits>

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// What a logit counts as: NaN as -inf (never above a number), +inf as the
// largest finite value (so that the softmax stays defined).
__device__ __forceinline__ float clean(float l) {
  return fminf(fmaxf(l, -INFINITY), FLT_MAX);  // fmaxf gives the operand that is no NaN
}

__device__ __forceinline__ double shfl_xor_f64(double v, int mask) {
  return __shfl_xor(v, mask, kWave);
}

struct RouteArgs {
  const float* logits;
  const float* bias;  // or nullptr
  int64_t T;
  int E, k;
  int groups, top_groups;  // groups 1 when every group is kept
  int size;                // experts of a group, E / groups
  int lpg, cpl;            // lanes of a group, experts of a lane
  bool sigmoid, top2, renorm;
  bool vec, full;  // loads of four experts; every lane has VPL of them
  float scale;
  int32_t* idx;
  float* w;
};

// Max and min over the G lanes of a group, in every lane of it: exchanges
// inside 16-lane rows by DPP, across rows by the row and half swaps.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return static_cast<int>(
      __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xF, 0xF, false);
}
template <int G, class T, class F>
__device__ __forceinline__ T group_reduce(T v, F&& f) {
  static_assert(G == 8 || G == 16 || G == 32 || G == 64, "lanes of a token");
  if constexpr (G >= 16) {
    v = f(v, dpp<0x128>(v));  // row_ror:8
    v = f(v, dpp<0x124>(v));  // row_ror:4
  } else {
    v = f(v, dpp<0x141>(v));  // row_half_mirror
  }
  v = f(v, dpp<0x4E>(v));  // quad_perm [2,3,0,1]
  v = f(v, dpp<0xB1>(v));  // quad_perm [1,0,3,2]
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v),
                                                    __builtin_bit_cast(uint32_t, v), false, false);
    v = f(__builtin_bit_cast(T, static_cast<uint32_t>(r[0])), __builtin_bit_cast(T, static_cast<uint32_t>(r[1])));
  }
  if constexpr (G == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v),
                                                    __builtin_bit_cast(uint32_t, v), false, false);
    v = f(__builtin_bit_cast(T, static_cast<uint32_t>(r[0])), __builtin_bit_cast(T, static_cast<uint32_t>(r[1])));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ float group_min(float v) {
  return group_reduce<G>(v, [](float a, float b) { return fminf(a, b); });
}
template <int G>
__device__ __forceinline__ int group_min(int v) {
  return group_reduce<G>(v, [](int a, int b) { return min(a, b); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// The largest value over the G lanes of a group, the lower expert among equals.
template <int G>
__device__ __forceinline__ void group_best(double& v, int& e) {
  auto take = [&](double ov, int oe) {
    if (ov > v || (ov == v && oe < e)) v = ov, e = oe;
  };
  auto step = [&](auto ctrl) {
    constexpr int CTRL = decltype(ctrl)::value;
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp<CTRL>(static_cast<uint32_t>(b)), hi = dpp<CTRL>(static_cast<uint32_t>(b >> 32));
    take(__builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo), dpp<CTRL>(e));
  };
  if constexpr (G >= 16) {
    step(std::integral_constant<int, 0x128>{});  // row_ror:8
    step(std::integral_constant<int, 0x124>{});  // row_ror:4
  } else {
    step(std::integral_constant<int, 0x141>{});  // row_half_mirror
  }
  step(std::integral_constant<int, 0x4E>{});  // quad_perm [2,3,0,1]
  step(std::integral_constant<int, 0xB1>{});  // quad_perm [1,0,3,2]
#pragma unroll
  for (int off = 16; off < G; off <<= 1) take(shfl_xor_f64(v, off), __shfl_xor(e, off, kWave));
}

// Where a lane's experts lie: [e0, e0 + n) of group grp.
struct Share {
  int j, grp, e0, n;
};

// The choice from fp64 scores, lane r of the group keeping the r-th expert.
template <int G, int VPL>
__device__ __forceinline__ int choose_exact(const RouteArgs& a, const float* row, Share sh) {
  double v[VPL];  // scores, then selection values
  float lmax = -INFINITY;
  float l[VPL];
#pragma unroll
  for (int q = 0; q < VPL; ++q) {
    l[q] = q < sh.n ? clean(row[sh.e0 + q]) : -INFINITY;
    lmax = fmaxf(lmax, l[q]);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int q = 0; q < VPL; ++q) v[q] = 1.0 / (1.0 + exp(-double(l[q])));
  } else {
    lmax = group_max<G>(lmax);
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < VPL; ++q) {
      v[q] = l[q] == -INFINITY ? 0.0 : exp(double(l[q]) - double(lmax));
      sum += v[q];
    }
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) sum += shfl_xor_f64(sum, off);
    if (sum == 0.0) sum = 1.0;  // no expert has a finite logit: every score is 0
#pragma unroll
    for (int q = 0; q < VPL; ++q) v[q] /= sum;
  }
  if (a.bias) {
#pragma unroll
    for (int q = 0; q < VPL; ++q)
      if (q < sh.n) {
        v[q] += double(a.bias[sh.e0 + q]);
        if (v[q] != v[q]) v[q] = -INFINITY;
      }
  }

  // open: the lane's experts that may still be selected
  uint32_t open = sh.n >= 32 ? 0xffffffffu : (1u << sh.n) - 1u;
  if (a.top_groups < a.groups) {
    double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int q = 0; q < VPL; ++q)
      if (q < sh.n) {
        m2 = fmax(m2, fmin(m1, v[q]));
        m1 = fmax(m1, v[q]);
      }
    for (int off = 1; off < a.lpg; off <<= 1) {
      const double o1 = shfl_xor_f64(m1, off), o2 = shfl_xor_f64(m2, off);
      m2 = fmax(fmin(m1, o1), fmax(m2, o2));
      m1 = fmax(m1, o1);
    }
    double rank = a.top2 && a.size > 1 ? m1 + m2 : m1;
    if (rank != rank) rank = -INFINITY;
    int place = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double r = __shfl(rank, g * a.lpg, G);
      place += (r > rank || (r == rank && g < sh.grp)) ? 1 : 0;
    }
    if (place >= a.top_groups) open = 0;
  }

  int my_e = 0;
  for (int r = 0; r < a.k; ++r) {
    double best = -INFINITY;
    int be = INT_MAX;
#pragma unroll
    for (int q = 0; q < VPL; ++q)
      if ((open >> q & 1u) && (v[q] > best || be == INT_MAX)) best = v[q], be = sh.e0 + q;
    group_best<G>(best, be);
    if (be >= sh.e0 && be < sh.e0 + sh.n) open &= ~(1u << (be - sh.e0));
    if (sh.j == r) my_e = be;
  }
  return my_e;
}

// A float's bits as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t ordered_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// A selection value as a 31-bit integer of the same order, its last bits giving
// way to the value's place in the lane, lowest place highest: a lane's keys all
// differ. (0 is left for a group that is out.)
template <int VPL>
struct Key {
  static constexpr uint32_t kPlaces = VPL <= 4 ? 3u : VPL <= 8 ? 7u : VPL <= 16 ? 15u : 31u;
  static __device__ __forceinline__ uint32_t make(float v, int q) {
    return ((ordered_bits(v) >> 1) & ~kPlaces) | (kPlaces - static_cast<uint32_t>(q));
  }
  static __device__ __forceinline__ int place(uint32_t k) {
    return static_cast<int>(kPlaces - (k & kPlaces));
  }
};

template <int G, int VPL>
__global__ __launch_bounds__(kThreads) void route_scored_kernel(RouteArgs a) {
  const int64_t t_raw = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / G;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // idle groups repeat the last token, storing nothing
  const float* row = a.logits + t * a.E;
  Share sh;
  sh.j = threadIdx.x % G;
  sh.grp = sh.j / a.lpg;
  const int i0 = (sh.j % a.lpg) * a.cpl;  // first expert of the lane inside its group
  sh.n = sh.grp < a.groups ? max(0, min(a.cpl, a.size - i0)) : 0;
  sh.e0 = sh.grp * a.size + i0;
  const int j = sh.j;

  // fp32 scores, then selection values; -inf where there is no expert
  float v[VPL], b[VPL];
  if (a.vec) {  // every lane's experts start 16-byte aligned, in whole fours
#pragma unroll
    for (int q = 0; q < VPL; q += 4) {
      const int at = q < sh.n ? sh.e0 + q : 0;
      const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(row + at));
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
      if (a.bias) y = *reinterpret_cast<const f32x4*>(a.bias + at);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[q + u] = x[u], b[q + u] = y[u];
    }
  } else {
#pragma unroll
    for (int q = 0; q < VPL; ++q) {
      const int at = q < sh.n ? sh.e0 + q : 0;
      v[q] = row[at];
      b[q] = a.bias ? a.bias[at] : 0.f;
    }
  }
  // What a score may be off. Sigmoid: e^-l within (1 + 1.5 |l|) 2^-23 of itself
  // (the hardware's exponential and its argument), times s (1 - s), and the
  // reciprocal and sum, 2 * 2^-23: below 2^-21.4. Softmax, of the score itself: expf
  // and the product 3 half steps, the argument's rounding |l - max| half steps, and
  // the same factor 1 / sum for all: its terms' mean |l - max| (below 8 for
  // 1024 experts) and at most 38 additions matter only beside a bias.
  float lmax = -INFINITY, sum = 1.f, inv = 1.f;
  if (a.sigmoid) {
#pragma unroll
    for (int q = 0; q < VPL; ++q)  // NaN as -inf; e^-inf is 0 without clamping
      v[q] = __builtin_amdgcn_rcpf(1.f + __expf(-fmaxf(v[q], -INFINITY)));
  } else {
#pragma unroll
    for (int q = 0; q < VPL; ++q) {
      v[q] = q < sh.n ? clean(v[q]) : -INFINITY;
      lmax = fmaxf(lmax, v[q]);
    }
    lmax = group_max<G>(lmax);
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < VPL; ++q) {
      v[q] = v[q] == -INFINITY ? 0.f : expf(v[q] - lmax);
      sum += v[q];
    }
    sum = group_sum<G>(sum);
    if (sum == 0.f) sum = 1.f;  // no expert has a finite logit: every score is 0
    inv = 1.f / sum;
#pragma unroll
    for (int q = 0; q < VPL; ++q) v[q] *= inv;
  }
#pragma unroll
  for (int q = 0; q < VPL; ++q) v[q] = fmaxf(v[q] + b[q], -INFINITY);
  if (!a.full) {
#pragma unroll
    for (int q = 0; q < VPL; ++q) v[q] = q < sh.n ? v[q] : -INFINITY;
  }

  bool sure = true, keep = true;
  if (a.top_groups < a.groups) {
    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int q = 0; q < VPL; ++q) {
      m2 = fmaxf(m2, fminf(m1, v[q]));
      m1 = fmaxf(m1, v[q]);
    }
    for (int off = 1; off < a.lpg; off <<= 1) {
      const float o1 = __shfl_xor(m1, off, kWave), o2 = __shfl_xor(m2, off, kWave);
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    }
    const float rank = fmaxf(a.top2 && a.size > 1 ? m1 + m2 : m1, -INFINITY);
    // the ranks as integers, their last bits giving way to the group (lower first); an order
    // that the bits left out would have turned shows below as lowest < highest
    const uint32_t mine = (ordered_bits(rank) & ~63u) | (63u - static_cast<uint32_t>(sh.grp));
    int place = 0;
    for (int g = 0; g < a.groups; ++g)
      place += static_cast<uint32_t>(__shfl(static_cast<int>(mine), g * a.lpg, G)) > mine ? 1 : 0;
    const bool in = sh.grp < a.groups;
    keep = in && place < a.top_groups;
    const float lowest = group_min<G>(keep ? rank : INFINITY);
    const float highest = group_max<G>(in && !keep ? rank : -INFINITY);
    // A rank's error: its scores', and half a step for each sum of fp32 values, of the
    // two values' own size (which may cancel: a rank can be far smaller than they are). A
    // rank of -inf is exact. (Softmax: no score is above 1 / sum; not greater:
    // infinities too are left to the exact choice.)
    const float terms = a.top2 && a.size > 1 ? fabsf(m1) + fabsf(m2) : fabsf(m1);
    const float off = a.sigmoid ? 0x1p-19f : (a.bias ? 0x1p-15f * inv : 0x1p-16f * lowest) + 0x1p-126f;
    sure = lowest - highest > off + 0x1p-20f * group_max<G>(in && rank > -INFINITY ? terms : 0.f);
  }

  // The k largest keys, and the one after them (unless there is no expert left). A
  // lane's next key is its largest below the one it gave last: the largest
  // key - last in 32-bit arithmetic, which the keys below `last`, and they alone,
  // wrap into the upper half. Equal keys of two lanes: the lower expert. (A place
  // without an expert is -inf; a choice of -inf is left to the exact choice.)
  uint32_t key[VPL], last = 0x80000000u;
  const uint32_t cap = keep ? 0x7fffffffu : 0u;
#pragma unroll
  for (int q = 0; q < VPL; ++q) key[q] = Key<VPL>::make(v[q], q);
  // Lane r keeps the r-th, r <= k: one more than is asked for; `beyond` is the one after that.
  const int candidates = a.top_groups * a.size, rounds = min(candidates, a.k + 2);
  int my_e = 0, beyond = 0;
  uint32_t lowest_key = 0;
  for (int r = 0; r < rounds; ++r) {
    uint32_t best = 0u - last;  // none left: 0
#pragma unroll
    for (int q = 0; q < VPL; ++q) best = max(best, key[q] - last);
    best = min(best + last, cap);
    const uint32_t top = group_max<G>(best);
    const int e = group_min<G>(best == top ? sh.e0 + Key<VPL>::place(best) : INT_MAX);
    last = best == top && e == sh.e0 + Key<VPL>::place(best) ? best : last;
    if (j == r) my_e = e;
    beyond = e;
    lowest_key = top;
  }
  sure = sure && lowest_key > (Key<VPL>::make(-INFINITY, 0) | Key<VPL>::kPlaces);
  my_e = min(my_e, a.E - 1), beyond = min(beyond, a.E - 1);

  // The candidates' values again, each from its own logit, against the next one's:
  // far enough apart (or a true tie), or `near`. The keys order values of which they leave
  // out the last bits, at most 2^-17 of a value: `beyond`, and all that was not
  // looked at, has to lie that much (of both) below the k-th.
  const bool mine = j < a.k, held = j < min(rounds, a.k + 1);
  bool near = false;
  const float lj = clean(row[my_e]);
  const float bj = a.bias ? a.bias[my_e] : 0.f;
  {
    // a logit's selection value, and by how much it may be off
    auto value = [&](float l, float bias, float& off) {
      float x, far;
      if (a.sigmoid) {
        x = __builtin_amdgcn_rcpf(1.f + __expf(-l));
        off = 0x1p-21f;
      } else {
        far = lmax - l;
        x = (l == -INFINITY ? 0.f : expf(-far)) * inv;
        // (below the normal range the roundings, and the bits that a key leaves out, are whole
        // smallest steps, 2^-143 at most; a score that is 0 by its formula is exact)
        off = l > -INFINITY ? x * ((a.bias ? 64.f : 8.f) + far) * 0x1p-24f + 0x1p-126f : 0.f;
      }
      const float v = fmaxf(x + bias, -INFINITY);
      off += 0x1p-23f * fabsf(v);
      return v;
    };
    float off_j, off_b;
    const float vj = value(lj, bj, off_j);
    const float vb = value(clean(row[beyond]), a.bias ? a.bias[beyond] : 0.f, off_b);
    const float l2 = __shfl_down(lj, 1, G), b2 = __shfl_down(bj, 1, G), v2 = __shfl_down(vj, 1, G),
                off_2 = __shfl_down(off_j, 1, G);
    if (held) sure = sure && vj > -INFINITY;
    const int e2 = __shfl_down(my_e, 1, G);
    // (a true tie may stand in the order of the places in two lanes)
    if (mine && j + 1 < rounds)
      near = !(vj - v2 > off_j + off_2 || (lj == l2 && bj == b2 && my_e < e2));
    if (j + 1 == a.k && rounds == a.k + 2)
      sure = sure && vj - vb > off_j + off_b + 0x1.8p-17f * (fabsf(vj) + fabsf(vb));
  }
  float ls = lj;
  if (__any(!sure) || (!a.sigmoid && a.bias && __any(near))) {
    // one such token: the wavefront's tokens all choose again (the same, where they were sure)
    my_e = choose_exact<G, VPL>(a, row, sh);
    ls = clean(row[my_e]);
  } else if (__any(near)) {
    // the candidates are the right ones, their order is that of their fp64 values
    // (softmax: without its common factor; 0 at -inf, also where lmax is -inf itself)
    const double v = a.sigmoid         ? 1.0 / (1.0 + exp(-double(lj))) + double(bj)
                     : lj == -INFINITY ? 0.0
                                       : exp(double(lj) - double(lmax));
    int place = 0;
    for (int i = 0; i < min(rounds, a.k + 1); ++i) {
      const double vi = __shfl(v, i, G);
      const int ei = __shfl(my_e, i, G);
      place += (vi > v || (vi == v && ei < my_e)) ? 1 : 0;
    }
    // each to its place; lanes that hold none to their own
    const int to = (lane_id() & ~(G - 1)) + (held ? place : j);
    my_e = __builtin_amdgcn_ds_permute(to * 4, my_e);
    ls = clean(row[my_e]);
  }

  // The weights, from the selected logits, in fp64 up to their one rounding (an exponential
  // a lane; in fp32 they were a second half step off, and 65536 tokens no faster).
  // Only the softmax's sum over all experts is one of fp32 terms.
  float top = lmax;
  if (!a.sigmoid && a.renorm) top = group_max<G>(mine ? ls : -INFINITY);  // of the selected alone
  double s = 0.0;
  if (mine && ls > -INFINITY)
    s = a.sigmoid ? 1.0 / (1.0 + exp(-double(ls))) : exp(double(ls) - double(top));
  double total = s;
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) total += shfl_xor_f64(total, off);
  if (!a.renorm) total = double(sum);  // 1 for the sigmoid
  const float w = total == 0.0 ? 0.f : static_cast<float>(s / total * double(a.scale));
  if (live && mine) {
    a.idx[t * a.k + j] = my_e;
    a.w[t * a.k + j] = w;
  }
}

// The gradient of the weights with respect to the logits; the choice itself
// (and so the bias) has none. With g = grad_w and p the scores:
//
//   sigmoid:            dl_j = scale * g_j p_j (1 - p_j)
//   sigmoid, renorm:    dl_j = scale * (g_j - sum_i g_i p_i / S) / S * p_j (1 - p_j),  S = sum_i p_i
//   softmax, renorm:    dl_j = scale * q_j (g_j - sum_i g_i q_i),  q the softmax of the selected logits
//   softmax:            dl_e = scale * p_e (g_e [e selected] - sum_i g_i p_i),   every e
//
// The last one's difference cancels for an expert that holds nearly all of its
// token: for a selected e it is formed as g_e (1 - p_e) - sum_{i != e} g_i p_i, with
// 1 - p_e of the largest from the sum of the others' terms.
//
// G lanes own a token. Lane j < k forms slot j's value (sums over the slots
// in fp64: they are few), the values are laid into an LDS row of E floats (over
// the unselected experts' own, where every logit has a gradient),
// and the lanes store the row four experts at a time. Bound by memory: 65536 tokens of
// 256 experts, softmax over all: 28 us, 4.9 TB/s.
struct RouteGradArgs {
  const float* logits;
  const int32_t* idx;
  const float* gw;
  int64_t T;
  int E, k;
  bool sigmoid, renorm;
  float scale;
  float* out;
};

template <int G>
__global__ __launch_bounds__(kThreads) void route_scored_grad_kernel(RouteGradArgs a) {
  constexpr int kQ = 4;  // chunks of four experts a lane holds at most: E <= 16 G
  __shared__ f32x4 tile[kThreads / G][G * kQ];
  const int slot = threadIdx.x / G, j = threadIdx.x % G;
  const int64_t t_raw = static_cast<int64_t>(blockIdx.x) * (kThreads / G) + slot;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;
  const float* row = a.logits + t * a.E;
  const int E = a.E, chunks = (E + 3) / 4;
  const bool full = !a.sigmoid && !a.renorm;  // every logit has a gradient
  const bool vec = (E & 3) == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;

  float l[kQ][4];
  float lmax = -INFINITY, sum = 1.f, rest = 0.f;  // rest: the terms of the sum that are not 1
  if (full) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int c = j + q * G;
      f32x4 x = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (c < chunks) {
        if (vec) {
          x = *reinterpret_cast<const f32x4*>(row + 4 * c);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (4 * c + u < E) x[u] = row[4 * c + u];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        l[q][u] = clean(x[u]);
        lmax = fmaxf(lmax, l[q][u]);
      }
    }
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) lmax = fmaxf(lmax, __shfl_xor(lmax, off, kWave));
    float ones = 0.f;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        l[q][u] = l[q][u] == -INFINITY ? 0.f : expf(l[q][u] - lmax);
        (l[q][u] == 1.f ? ones : rest) += l[q][u];
      }
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) {
      ones += __shfl_xor(ones, off, kWave);
      rest += __shfl_xor(rest, off, kWave);
    }
    sum = ones == 0.f ? 1.f : ones + rest;  // no expert has a finite logit: every score is 0
    rest += ones - 1.f;  // beside one of the largest
  }

  // slot j: its score, its gradient, and what it puts at its expert
  const int e = j < a.k ? a.idx[t * a.k + j] : -1;
  const bool ok = e >= 0 && e < E;
  const float lj = ok ? clean(row[e]) : -INFINITY;
  const double g = ok ? double(a.gw[t * a.k + j]) : 0.0;
  double p;
  if (a.sigmoid) {
    p = ok ? 1.0 / (1.0 + exp(-double(lj))) : 0.0;
  } else {
    float top = lmax;
    if (a.renorm) {
      top = lj;
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
    }
    p = lj == -INFINITY ? 0.0 : exp(double(lj) - double(top));
    if (!a.renorm) p /= double(sum);
  }
  double total = p, inner = g * p;
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) {
    total += shfl_xor_f64(total, off);
    inner += shfl_xor_f64(inner, off);
  }
  double d = 0.0;
  if (full) {
    // from g and the others' g p, below
  } else if (a.sigmoid) {
    const double slope = ok ? p / (1.0 + exp(double(lj))) : 0.0;  // p (1 - p)
    d = (a.renorm ? (total == 0.0 ? 0.0 : (g - inner / total) / total) : g) * slope;
  } else {
    d = total == 0.0 ? 0.0 : p / total * (g - inner / total);
  }
  if (!full) d *= double(a.scale);

  // a repeated expert takes the sum of its slots, in slot order, at the first of them
  double dsum = 0.0;
  bool first = true;
  if (full) {
    const float g32 = static_cast<float>(g), gp32 = static_cast<float>(g * p);
    double others = 0.0;
    for (int i = 0; i < a.k; ++i) {
      const int ei = __shfl(e, i, G);
      const float gi = __shfl(g32, i, G), gpi = __shfl(gp32, i, G);
      if (ei == e) {
        dsum += double(gi);
        if (i < j) first = false;
      } else {
        others += double(gpi);
      }
    }
    const bool one = lj > -INFINITY && expf(lj - lmax) == 1.f;
    const double left = one ? double(rest / sum) : 1.0 - p;
    dsum = double(a.scale) * p * (dsum * left - others);
  } else {
    for (int i = 0; i < a.k; ++i) {
      const int ei = __shfl(e, i, G);
      const double di = __shfl(d, i, G);
      if (ei == e) {
        dsum += di;
        if (i < j) first = false;
      }
    }
  }

  const float factor = a.scale / sum, fi = static_cast<float>(inner);
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (j + q * G >= chunks) continue;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (full) {
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = factor * l[q][u] * (0.f - fi);
    }
    tile[slot][j + q * G] = x;
  }
  __syncthreads();
  if (ok && first) reinterpret_cast<float*>(tile[slot])[e] = static_cast<float>(dsum);
  __syncthreads();
  if (!live) return;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int c = j + q * G;
    if (c >= chunks) continue;
    const f32x4 x = tile[slot][c];
    float* o = a.out + t * E + 4 * c;
    if (vec) {
      __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(o));
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (4 * c + u < E) o[u] = x[u];
    }
  }
}

template <int G, int VPL>
bool fits(int k, int groups, int size, int& lpg, int& cpl) {
  if (k >= G || groups > G) return false;  // lane k holds the first candidate left out
  lpg = 1;
  while (lpg * 2 * groups <= G) lpg *= 2;
  cpl = (size + lpg - 1) / lpg;
  return cpl <= VPL;
}

template <int G, int VPL>
bool launch(RouteArgs a, hipStream_t s) {
  if (!fits<G, VPL>(a.k, a.groups, a.size, a.lpg, a.cpl)) return false;
  // fours of experts that neither a lane nor a group splits
  const bool fours = a.size % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.bias)) & 15) == 0;
  if (fours) a.cpl = (a.cpl + 3) / 4 * 4;
  a.vec = fours && a.cpl <= VPL;
  if (!a.vec) a.cpl = (a.size + a.lpg - 1) / a.lpg;
  a.full = a.cpl == VPL && a.size == a.lpg * VPL && a.groups * a.lpg == G;
  const int64_t per = kThreads / G;
  route_scored_kernel<G, VPL>
      <<<dim3(static_cast<unsigned>((a.T + per - 1) / per)), kThreads, 0, s>>>(a);
  return true;
}

template <int G>
void launch_grad(const RouteGradArgs& a, hipStream_t s) {
  const int64_t per = kThreads / G;
  route_scored_grad_kernel<G>
      <<<dim3(static_cast<unsigned>((a.T + per - 1) / per)), kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_route_scored(const moe_route_desc& d, const float* logits, const float* bias,
                               int32_t* idx, float* w, hipStream_t s) {
  RouteArgs a{};
  a.logits = logits, a.bias = bias, a.T = d.num_tokens, a.E = d.num_experts, a.k = d.top_k;
  // keeping every group is the same as having one
  a.groups = d.top_groups < d.num_groups ? d.num_groups : 1;
  a.top_groups = a.groups == 1 ? 1 : d.top_groups;
  a.size = a.E / a.groups;
  a.sigmoid = d.score == MOE_SCORE_SIGMOID, a.top2 = d.group_rank == MOE_GROUP_TOP2;
  a.renorm = d.renormalise != 0, a.scale = d.scale;
  a.idx = idx, a.w = w;
  // The fewest lanes to a token that still give every SIMD four wavefronts, at 16
  // experts to a lane at most: with many tokens a wavefront shares its exchanges
  // among up to eight of them (65536 tokens of 256 experts: 16 lanes 46 us, 32 lanes 51 us; of 128
  // experts: 8 lanes 27 us, 32 lanes 47 us), with few each token's chain of steps is what is waited
  // for (16 tokens of 256: 64 lanes 5.5 us, 16 lanes 15 us). 32 experts to a lane
  // read 128 bytes apart and took 74 us.
  const int64_t lanes = int64_t(16) * kWave * device_cu_count() / a.T;
  const bool done = (lanes <= 8 && (launch<8, 8>(a, s) || launch<8, 16>(a, s))) ||
                    (lanes <= 16 && (launch<16, 8>(a, s) || launch<16, 16>(a, s))) ||
                    (lanes <= 32 && (launch<32, 8>(a, s) || launch<32, 16>(a, s))) ||
                    launch<64, 4>(a, s) || launch<64, 16>(a, s) || launch<64, 32>(a, s);
  if (!done) return hipErrorInvalidValue;  // not reached: groups <= 64 and E <= 1024 fit the last
  return hipGetLastError();
}

hipError_t launch_route_scored_backward(const moe_route_desc& d, const float* logits,
                                        const int32_t* idx, const float* gw, float* out,
                                        hipStream_t s) {
  RouteGradArgs a{logits, idx, gw, d.num_tokens, d.num_experts, d.top_k,
                  d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, d.scale, out};
  if (a.E <= 128 && a.k <= 8) launch_grad<8>(a, s);
  else if (a.E <= 256) launch_grad<16>(a, s);
  else if (a.E <= 512) launch_grad<32>(a, s);
  else launch_grad<64>(a, s);
  return hipGetLastError();
}

}  // namespace moe
