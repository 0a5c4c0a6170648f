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
// The scores that decide a choice are formed in fp64: an fp32 sigmoid rounds
// by up to 2^-24, and at 65536 tokens of 256 experts a few tokens have two
// candidates closer than that, so fp32 scores would choose by rounding.
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
  return l != l ? -INFINITY : fminf(l, FLT_MAX);
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
  float scale;
  int32_t* idx;
  float* w;
};

template <int G, int VPL>
__global__ __launch_bounds__(kThreads) void route_scored_kernel(RouteArgs a) {
  const int64_t t_raw = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / G;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // idle groups repeat the last token, storing nothing
  const int j = threadIdx.x % G;
  const float* row = a.logits + t * a.E;

  const int grp = j / a.lpg;
  const int i0 = (j % a.lpg) * a.cpl;  // first expert of the lane inside its group
  const int n = grp < a.groups ? max(0, min(a.cpl, a.size - i0)) : 0;
  const int e0 = grp * a.size + i0;

  double v[VPL];  // scores, then selection values
  float lmax = -INFINITY;
  float l[VPL];
#pragma unroll
  for (int q = 0; q < VPL; ++q) {
    l[q] = q < n ? clean(row[e0 + q]) : -INFINITY;
    lmax = fmaxf(lmax, l[q]);
  }
  double sum = 1.0;
  if (a.sigmoid) {
#pragma unroll
    for (int q = 0; q < VPL; ++q) v[q] = 1.0 / (1.0 + exp(-double(l[q])));
  } else {
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) lmax = fmaxf(lmax, __shfl_xor(lmax, off, kWave));
    sum = 0.0;
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
      if (q < n) {
        v[q] += double(a.bias[e0 + q]);
        if (v[q] != v[q]) v[q] = -INFINITY;
      }
  }

  // open: the lane's experts that may still be selected
  uint32_t open = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  if (a.top_groups < a.groups) {
    double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int q = 0; q < VPL; ++q)
      if (q < n) {
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
      place += (r > rank || (r == rank && g < grp)) ? 1 : 0;
    }
    if (place >= a.top_groups) open = 0;
  }

  int my_e = 0;
  for (int r = 0; r < a.k; ++r) {
    double best = -INFINITY;
    int be = INT_MAX;
#pragma unroll
    for (int q = 0; q < VPL; ++q)
      if ((open >> q & 1u) && (v[q] > best || be == INT_MAX)) best = v[q], be = e0 + q;
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) {
      const double ob = shfl_xor_f64(best, off);
      const int oe = __shfl_xor(be, off, kWave);
      if (ob > best || (ob == best && oe < be)) best = ob, be = oe;
    }
    if (be >= e0 && be < e0 + n) open &= ~(1u << (be - e0));
    if (j == r) my_e = be;
  }

  // weights of the selected experts, from their logits
  const bool mine = j < a.k;
  const float lj = mine ? clean(row[my_e]) : -INFINITY;
  double s;
  if (a.sigmoid) {
    s = mine ? 1.0 / (1.0 + exp(-double(lj))) : 0.0;
  } else {
    float top = lmax;
    if (a.renorm) {  // the softmax of the selected logits alone
      top = lj;
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
    }
    s = lj == -INFINITY ? 0.0 : exp(double(lj) - double(top));
    if (!a.renorm) s /= sum;
  }
  if (a.renorm) {
    double total = s;
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) total += shfl_xor_f64(total, off);
    s = total == 0.0 ? 0.0 : s / total;
  }
  if (live && mine) {
    a.idx[t * a.k + j] = my_e;
    a.w[t * a.k + j] = static_cast<float>(s * double(a.scale));
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
// G lanes own a token. Lane j < k forms slot j's value (sums over the slots
// in fp64: they are few), the values are laid into an LDS row of E floats,
// and the lanes store the row four experts at a time.
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
  float lmax = -INFINITY, sum = 1.f;
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
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        l[q][u] = l[q][u] == -INFINITY ? 0.f : expf(l[q][u] - lmax);
        sum += l[q][u];
      }
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, kWave);
    if (sum == 0.f) sum = 1.f;
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
  double d;
  if (full) {
    d = g;  // the row below scales it by the expert's own score
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
  for (int i = 0; i < a.k; ++i) {
    const int ei = __shfl(e, i, G);
    const double di = __shfl(d, i, G);
    if (ei == e) {
      dsum += di;
      if (i < j) first = false;
    }
  }

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < kQ; ++q)
    if (j + q * G < chunks) tile[slot][j + q * G] = zero;
  __syncthreads();
  if (ok && first) reinterpret_cast<float*>(tile[slot])[e] = static_cast<float>(dsum);
  __syncthreads();
  if (!live) return;
  const float factor = a.scale / sum, fi = static_cast<float>(inner);
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int c = j + q * G;
    if (c >= chunks) continue;
    f32x4 x = tile[slot][c];
    if (full) {
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = factor * l[q][u] * (x[u] - fi);
    }
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
  if (k > G || groups > G) return false;
  lpg = 1;
  while (lpg * 2 * groups <= G) lpg *= 2;
  cpl = (size + lpg - 1) / lpg;
  return cpl <= VPL;
}

template <int G, int VPL>
void launch(const RouteArgs& a, hipStream_t s) {
  const int64_t per = kThreads / G;
  route_scored_kernel<G, VPL>
      <<<dim3(static_cast<unsigned>((a.T + per - 1) / per)), kThreads, 0, s>>>(a);
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
  // the fewest lanes a token's experts fit: more tokens to a wavefront share its exchanges
  if (fits<8, 8>(a.k, a.groups, a.size, a.lpg, a.cpl)) launch<8, 8>(a, s);
  else if (fits<16, 8>(a.k, a.groups, a.size, a.lpg, a.cpl)) launch<16, 8>(a, s);
  else if (fits<16, 16>(a.k, a.groups, a.size, a.lpg, a.cpl)) launch<16, 16>(a, s);
  else if (fits<32, 16>(a.k, a.groups, a.size, a.lpg, a.cpl)) launch<32, 16>(a, s);
  else if (fits<64, 16>(a.k, a.groups, a.size, a.lpg, a.cpl)) launch<64, 16>(a, s);
  else if (fits<64, 32>(a.k, a.groups, a.size, a.lpg, a.cpl)) launch<64, 32>(a, s);
  else return hipErrorInvalidValue;  // not reached: groups <= 64 and E <= 1024 fit the last
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
