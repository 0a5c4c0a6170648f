// Root-mean-square norm with the residual's addition, its output in the rows'
// type and/or in 8 bits with scales, and its gradients.
//
//   forward   h = x + residual, rounded to the rows' type
//             y = h rstd gain,  rstd = 1 / sqrt(mean(h^2) + eps)
//   backward  dh = rstd (gain dy - xhat mean(gain dy xhat)) + dtotal,  xhat = h rstd
//             dgain = sum over rows of dy xhat
//
// One pass over the data: WAVES wavefronts hold a row in registers between the
// sum of squares and the outputs, eight values of consecutive columns to a lane,
// so that 16 neighbouring lanes hold the 128 values of a scale. Sums are fp32;
// y is fp32 until its one rounding to each output. The backward takes both sums
// of a row together (mean(h^2) and mean(gain dy h)), so it needs no statistics
// kept by the forward. dgain: a lane keeps its columns' sums over all of its
// workgroup's rows, the workgroups' sums are added in order by a second launch
// (fp64), so that the result does not depend on timing.
// Bound: HBM. A workgroup walks several rows and keeps the gain in registers.
// 65536 x 7168 bf16 with residual, total and 8-bit output: 615 us, 5.4 TB/s (a large copy
// reaches 4.9); the gradients of 16384 x 7168: 186 us, 5.0 TB/s.
#include <algorithm>

#include "../../include/moe.h"
#include "fp8.h"

namespace moe {
namespace {

struct NormArgs {
  const void* x;
  const void* residual;  // or nullptr
  const float* gain;     // or nullptr: ones
  void* total;           // or nullptr
  void* y;               // or nullptr
  void* q;               // or nullptr: [rows, H] e4m3
  float* scale;          // [rows, runs]
  int64_t rows, ldx, ldr, ldt, ldy;
  int H, runs;
  float eps;
};

__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

// The row's sums over all of its wavefronts, the same bits in each of them.
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int wid) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WAVES > 1) {
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * WAVES + wid] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v[i] += red[i * WAVES + w];
    }
  }
}

template <int VPT>
__device__ __forceinline__ void load_gain(const float* gain, int H, int c0, int step,
                                          float (&g)[VPT][8]) {
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (c0 + i * step) * 8;
    f32x4 a{1.f, 1.f, 1.f, 1.f}, b = a;
    if (gain && c < H) {
      a = *reinterpret_cast<const f32x4*>(gain + c);
      b = *reinterpret_cast<const f32x4*>(gain + c + 4);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) g[i][j] = a[j], g[i][4 + j] = b[j];
  }
}

// rows of a workgroup at a time: one per WAVES wavefronts
template <int WAVES>
constexpr int block_waves() { return WAVES < 4 ? 4 : WAVES; }

template <int T, int WAVES, int VPT>
__global__ __launch_bounds__(64 * block_waves<WAVES>()) void norm_kernel(NormArgs a) {
  constexpr int BW = block_waves<WAVES>(), PER = BW / WAVES, LANES = 64 * WAVES;
  // two sets, a row apart: a wavefront may be at the next row while another still adds this one
  __shared__ float red[2][BW];
  const int wid = threadIdx.x / 64, sub = wid / WAVES;
  const int c0 = threadIdx.x % LANES;
  float g[VPT][8];
  load_gain<VPT>(a.gain, a.H, c0, LANES, g);
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * PER + sub; row < a.rows;
       row += int64_t(gridDim.x) * PER, turn ^= 1) {
    Raw<T> rx[VPT], rr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (c0 + i * LANES) * 8;
      if (c < a.H) {
        rx[i] = load8<T>(a.x, row * a.ldx + c);
        if (a.residual) rr[i] = load8<T>(a.residual, row * a.ldr + c);
      }
    }
    float h[VPT][8], sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (c0 + i * LANES) * 8;
      if (c < a.H) {
        values8<T>(rx[i], h[i]);
        if (a.residual) {
          float r[8];
          values8<T>(rr[i], r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[j];
          const Raw<T> t = raw8<T>(h[i]);
          if (a.total) store8<T>(a.total, row * a.ldt + c, t);
          values8<T>(t, h[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] += h[i][j] * h[i][j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      }
    }
    row_sums<WAVES>(sum, red[turn] + sub * WAVES, wid % WAVES);
    const float rstd = 1.f / sqrtf(sum[0] / float(a.H) + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (c0 + i * LANES) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = c < a.H ? h[i][j] * rstd * g[i][j] : 0.f;
      if (a.q) {
        const float s = scale_of(max16(magnitude(h[i])));
        if (c < a.H) {
          store_fp8x8(a.q, row * a.H + c, to_fp8x8(h[i], 1.f / s));
          if ((c & (kRun - 1)) == 0) a.scale[row * a.runs + c / kRun] = s;
        }
      }
      if (a.y && c < a.H) store8<T>(a.y, row * a.ldy + c, raw8<T>(h[i]));
    }
  }
}

struct NormGradArgs {
  const void* dy;
  const void* h;
  const float* gain;
  const void* dtotal;  // or nullptr
  void* dh;            // or nullptr
  float* sums;         // [gridDim.x, H] or nullptr
  int64_t rows, ldy, ldh, ldt, ldd;
  int H;
  float eps;
};

template <int T, int WAVES, int VPT>
__global__ __launch_bounds__(64 * block_waves<WAVES>()) void norm_grad_kernel(NormGradArgs a) {
  constexpr int BW = block_waves<WAVES>(), PER = BW / WAVES, LANES = 64 * WAVES;
  __shared__ float red[2][2 * BW];
  __shared__ float part[PER > 1 ? PER : 1][PER > 1 ? VPT * 512 : 1];
  const int wid = threadIdx.x / 64, sub = wid / WAVES;
  const int c0 = threadIdx.x % LANES;
  float g[VPT][8], dg[VPT][8];
  load_gain<VPT>(a.gain, a.H, c0, LANES, g);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.f;
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * PER + sub; row < a.rows;
       row += int64_t(gridDim.x) * PER, turn ^= 1) {
    Raw<T> rh[VPT], rd[VPT], rt[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (c0 + i * LANES) * 8;
      if (c < a.H) {
        rh[i] = load8<T>(a.h, row * a.ldh + c);
        rd[i] = load8<T>(a.dy, row * a.ldy + c);
        if (a.dtotal && a.dh) rt[i] = load8<T>(a.dtotal, row * a.ldt + c);
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if ((c0 + i * LANES) * 8 >= a.H) continue;
      float h[8], d[8];
      values8<T>(rh[i], h);
      values8<T>(rd[i], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[0] += h[j] * h[j];
        sum[1] += d[j] * g[i][j] * h[j];
      }
    }
    row_sums<WAVES>(sum, red[turn] + sub * 2 * WAVES, wid % WAVES);
    const float rstd = 1.f / sqrtf(sum[0] / float(a.H) + a.eps);
    const float mean = sum[1] * rstd / float(a.H);  // of gain dy xhat
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (c0 + i * LANES) * 8;
      if (c >= a.H) continue;
      float h[8], d[8], t[8];
      values8<T>(rh[i], h);
      values8<T>(rd[i], d);
      if (a.dtotal && a.dh) values8<T>(rt[i], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = h[j] * rstd;
        dg[i][j] += d[j] * xhat;
        h[j] = rstd * (g[i][j] * d[j] - xhat * mean);
        if (a.dtotal && a.dh) h[j] += t[j];
      }
      if (a.dh) store8<T>(a.dh, row * a.ldd + c, raw8<T>(h));
    }
  }
  if (!a.sums) return;
  if constexpr (PER > 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) part[sub][(i * 64 + c0) * 8 + j] = dg[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += 64 * BW) {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < PER; ++p) s += part[p][c];
      a.sums[int64_t(blockIdx.x) * a.H + c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (c0 + i * LANES) * 8;
      if (c >= a.H) continue;
      float* o = a.sums + int64_t(blockIdx.x) * a.H + c;
      *reinterpret_cast<f32x4*>(o) = f32x4{dg[i][0], dg[i][1], dg[i][2], dg[i][3]};
      *reinterpret_cast<f32x4*>(o + 4) = f32x4{dg[i][4], dg[i][5], dg[i][6], dg[i][7]};
    }
  }
}

// dgain[c] = the workgroups' sums, in a fixed order: 32 columns to a workgroup, whole lines of a
// sum's row to eight lanes, every 128th row to a lane. (768 sums of 7168: 6.3 us; 18 with half lines
// and 16 lanes to a column, whose batches of loads waited for each other.)
__global__ __launch_bounds__(1024) void gain_grad_kernel(const float* sums, int blocks, int H,
                                                         float* dgain) {
  __shared__ double part[16][32];
  const int c = (threadIdx.x & 7) * 4, q = threadIdx.x >> 3;
  const int n = int(blockIdx.x) * 32 + c;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (n < H) {
    constexpr int kBatch = 8;  // loads in flight together
    for (int b = q; b < blocks; b += 128 * kBatch) {
      f32x4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        x[u] = b + 128 * u < blocks ? *reinterpret_cast<const f32x4*>(sums + int64_t(b + 128 * u) * H + n)
                                    : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += double(x[u][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int off = 8; off < kWave; off <<= 1) s[i] += __shfl_xor(s[i], off, kWave);
    if (lane_id() < 8) part[threadIdx.x / kWave][c + i] = s[i];
  }
  __syncthreads();
  if (threadIdx.x < 32 && int(blockIdx.x) * 32 + int(threadIdx.x) < H) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += part[w][threadIdx.x];
    dgain[blockIdx.x * 32 + threadIdx.x] = static_cast<float>(t);
  }
}

// f(waves of a row, chunks of eight to a lane), both at compile time. few: up to two rows to a
// CU, where a row's own latency counts and 16 wavefronts have a wide one in flight at once
// (7168 wide, bf16, residual and 8-bit output: 16 rows 4.5 us, with 4 wavefronts 5.4, 256 rows 5.7 and 6.6;
// the backward 256 rows 16.8 and 17.3, but 2048 rows 44.4 and 40.5). Rows of up to 4096 gain nothing by
// them (2048 wide, 384 rows: 5.9 us, with 4 wavefronts 4.2).
template <class F>
hipError_t by_width(int H, bool few, F&& f) {
  using std::integral_constant;
  const int chunks = (H + 7) / 8;
  if (chunks <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (chunks <= 128) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (chunks <= 256) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (chunks <= 512) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (few && chunks <= 1024) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (chunks <= 1024) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
}

template <class F>
hipError_t by_type(int dtype, F&& f) {
  if (dtype == MOE_ROWS_F32) return f(std::integral_constant<int, 2>{});
  if (dtype == MOE_ROWS_F16) return f(std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, 0>{});
}

// Workgroups of the backward: their number is the length of dgain's second sum.
int grad_blocks(int64_t rows, int H) {
  const int per = H <= 1024 ? 4 : 1;  // rows of a workgroup at a time
  return static_cast<int>(std::min<int64_t>((rows + per - 1) / per, 768));
}

}  // namespace

hipError_t launch_rms_norm(const moe_norm_desc& d, const void* x, const void* residual,
                           const float* gain, void* total, void* y, void* q, float* scale,
                           hipStream_t s) {
  NormArgs a{x, residual, gain, total, y, q, scale, d.rows, d.ldx, d.ldr, d.ldt, d.ldy,
             d.hidden, (d.hidden + kRun - 1) / kRun, d.eps};
  const int64_t cus = device_cu_count();
  return by_type(d.dtype, [&](auto t) {
    return by_width(d.hidden, d.rows <= 2 * cus, [&](auto waves, auto vpt) {
      constexpr int W = decltype(waves)::value, BW = block_waves<W>();
      const int64_t groups = (d.rows + BW / W - 1) / (BW / W);
      const int grid = static_cast<int>(std::min<int64_t>(groups, cus * 32 / BW));
      norm_kernel<decltype(t)::value, W, decltype(vpt)::value><<<grid, 64 * BW, 0, s>>>(a);
      return hipGetLastError();
    });
  });
}

size_t rms_norm_backward_workspace_bytes(const moe_norm_desc& d) {
  return size_t(grad_blocks(d.rows, d.hidden)) * d.hidden * sizeof(float);
}

hipError_t launch_rms_norm_backward(const moe_norm_desc& d, const void* dy, const void* h,
                                    const float* gain, const void* dtotal, void* dh, float* dgain,
                                    void* ws, hipStream_t s) {
  const int grid = grad_blocks(d.rows, d.hidden);
  NormGradArgs a{dy, h, gain, dtotal, dh, dgain ? static_cast<float*>(ws) : nullptr,
                 d.rows, d.ldy, d.ldx, d.ldt, d.ldr, d.hidden, d.eps};
  if (grid) {
    const hipError_t e = by_type(d.dtype, [&](auto t) {
      return by_width(d.hidden, d.rows <= 2 * device_cu_count(), [&](auto waves, auto vpt) {
        constexpr int W = decltype(waves)::value, BW = block_waves<W>();
        norm_grad_kernel<decltype(t)::value, W, decltype(vpt)::value><<<grid, 64 * BW, 0, s>>>(a);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (!dgain) return hipSuccess;
  gain_grad_kernel<<<(d.hidden + 31) / 32, 1024, 0, s>>>(a.sums, grid, d.hidden, dgain);
  return hipGetLastError();
}

}  // namespace moe
