// Norm of many gradient tensors together, and scaling them down to a bound.
//
//   sumsq = sum over all tensors and elements of g^2
//   coef  = min(1, max_norm / (sqrt(sumsq) + 1e-6)),   out = g * coef
//
// Both passes stream the tensors: bound by memory, one launch for up to
// kTensors tensors (their addresses and sizes travel in the kernel's
// arguments, so nothing is copied to the device first). A tensor is cut into
// 64 KiB chunks; the workgroups walk the chunks of all tensors with a fixed
// stride, so long and short tensors share the chip and each sum has a fixed
// order. Squares are summed in fp64: 2^30 fp32 additions would lose digits,
// and fp32 squares overflow from 1.8e19 on.
#include <algorithm>
#include <vector>

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 112;      // of one launch (kernel arguments are limited to 4 KiB)
constexpr int kChunkVecs = 4096;   // 16-byte vectors of a chunk
constexpr int kPerThread = kChunkVecs / kThreads;
constexpr int kBatch = 8;          // vectors a thread has in flight

struct TensorTable {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t numel[kTensors];
  int first[kTensors + 1];  // first chunk of each tensor
  uint8_t type[kTensors];
  int n;
};

// which tensor a chunk belongs to
__device__ __forceinline__ int tensor_of(const TensorTable& t, int chunk) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int TYPE>
struct Elem {
  static constexpr int kPer = TYPE == MOE_ROWS_F32 ? 4 : 8;  // elements of a 16-byte vector
  using raw = typename std::conditional<TYPE == MOE_ROWS_F32, float, uint16_t>::type;
  static __device__ __forceinline__ float load(raw r) {
    if constexpr (TYPE == MOE_ROWS_F32) return r;
    else if constexpr (TYPE == MOE_ROWS_F16) return static_cast<float>(__builtin_bit_cast(_Float16, r));
    else return from_bf16(r);
  }
  static __device__ __forceinline__ raw store(float f) {
    if constexpr (TYPE == MOE_ROWS_F32) return f;
    else if constexpr (TYPE == MOE_ROWS_F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    else return to_bf16(f);
  }
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[kPer]) {
    if constexpr (TYPE == MOE_ROWS_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = load(static_cast<uint16_t>(v[i] & 0xffffu));
        f[2 * i + 1] = load(static_cast<uint16_t>(v[i] >> 16));
      }
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[kPer]) {
    u32x4 v;
    if constexpr (TYPE == MOE_ROWS_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = uint32_t(store(f[2 * i])) | uint32_t(store(f[2 * i + 1])) << 16;
    }
    return v;
  }
};

// The elements [at, at + count) of a chunk: whole 16-byte vectors where the
// addresses allow, single elements behind them (or throughout).
template <int TYPE>
__device__ __forceinline__ double chunk_sumsq(const void* in, int64_t at, int count) {
  using E = Elem<TYPE>;
  const auto* p = static_cast<const typename E::raw*>(in) + at;
  double s[2] = {0.0, 0.0};
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const u32x4* v = reinterpret_cast<const u32x4*>(p);
    const int vecs = count / E::kPer;
    done = vecs * E::kPer;
    for (int b = 0; b < kPerThread; b += kBatch) {
      u32x4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = (b + u) * kThreads + threadIdx.x;
        x[u] = i < vecs ? v[i] : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float f[E::kPer];
        E::unpack(x[u], f);
#pragma unroll
        for (int q = 0; q < E::kPer; ++q) s[q & 1] = fma(double(f[q]), double(f[q]), s[q & 1]);
      }
    }
  }
  for (int i = done + int(threadIdx.x); i < count; i += kThreads) {
    const double f = double(E::load(p[i]));
    s[0] = fma(f, f, s[0]);
  }
  return s[0] + s[1];
}

template <int TYPE>
__device__ __forceinline__ void chunk_scale(const void* in, void* out, int64_t at, int count,
                                            float coef) {
  using E = Elem<TYPE>;
  const auto* p = static_cast<const typename E::raw*>(in) + at;
  auto* o = static_cast<typename E::raw*>(out) + at;
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
    const u32x4* v = reinterpret_cast<const u32x4*>(p);
    u32x4* w = reinterpret_cast<u32x4*>(o);
    const int vecs = count / E::kPer;
    done = vecs * E::kPer;
    for (int b = 0; b < kPerThread; b += kBatch) {
      u32x4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = (b + u) * kThreads + threadIdx.x;
        if (i < vecs) x[u] = v[i];
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = (b + u) * kThreads + threadIdx.x;
        if (i < vecs) {
          float f[E::kPer];
          E::unpack(x[u], f);
#pragma unroll
          for (int q = 0; q < E::kPer; ++q) f[q] *= coef;
          __builtin_nontemporal_store(E::pack(f), w + i);
        }
      }
    }
  }
  for (int i = done + int(threadIdx.x); i < count; i += kThreads) o[i] = E::store(E::load(p[i]) * coef);
}

// Sum over the workgroup, in thread 0.
__device__ __forceinline__ double block_sum(double s, double* lds) {
#pragma unroll
  for (int off = kWave / 2; off >= 1; off >>= 1) s += __shfl_xor(s, off, kWave);
  if (lane_id() == 0) lds[threadIdx.x / kWave] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < int(blockDim.x) / kWave; ++w) s += lds[w];
  return s;
}

__device__ __forceinline__ int chunk_elems(int type) {
  return type == MOE_ROWS_F32 ? kChunkVecs * 4 : kChunkVecs * 8;
}

__global__ __launch_bounds__(kThreads) void sumsq_kernel(TensorTable t, double* part) {
  __shared__ double lds[kThreads / kWave];
  const int total = t.first[t.n];
  double s = 0.0;
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = uniform(tensor_of(t, c));
    const int type = t.type[i], per = chunk_elems(type);
    const int64_t at = int64_t(c - t.first[i]) * per;
    const int count = static_cast<int>(min(int64_t(per), t.numel[i] - at));
    if (type == MOE_ROWS_BF16) s += chunk_sumsq<MOE_ROWS_BF16>(t.in[i], at, count);
    else if (type == MOE_ROWS_F16) s += chunk_sumsq<MOE_ROWS_F16>(t.in[i], at, count);
    else s += chunk_sumsq<MOE_ROWS_F32>(t.in[i], at, count);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void sumsq_join_kernel(const double* part, int n, double* out) {
  __shared__ double lds[1024 / kWave];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) *out = s;
}

__global__ __launch_bounds__(kThreads) void clip_kernel(TensorTable t, const double* sumsq,
                                                        float max_norm, float* norm_out) {
  const double norm = sqrt(*sumsq);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
  const double ratio = double(max_norm) / (norm + 1e-6);
  // NaN stays NaN, but no bound leaves gradients of an infinite norm as they are
  const float coef = ratio >= 1.0 || (isinf(norm) && isinf(max_norm)) ? 1.0f : static_cast<float>(ratio);
  const int total = t.first[t.n];
  // from the end backwards: what the norm's pass read last may still be in the caches
  for (int c = total - 1 - int(blockIdx.x); c >= 0; c -= gridDim.x) {
    const int i = uniform(tensor_of(t, c));
    if (coef == 1.0f && t.in[i] == t.out[i]) continue;  // nothing changes in place
    const int type = t.type[i], per = chunk_elems(type);
    const int64_t at = int64_t(c - t.first[i]) * per;
    const int count = static_cast<int>(min(int64_t(per), t.numel[i] - at));
    if (type == MOE_ROWS_BF16) chunk_scale<MOE_ROWS_BF16>(t.in[i], t.out[i], at, count, coef);
    else if (type == MOE_ROWS_F16) chunk_scale<MOE_ROWS_F16>(t.in[i], t.out[i], at, count, coef);
    else chunk_scale<MOE_ROWS_F32>(t.in[i], t.out[i], at, count, coef);
  }
}

int64_t elem_bytes(int type) { return type == MOE_ROWS_F32 ? 4 : 2; }

int64_t chunks_of(const moe_tensor_ref& r) {
  const int64_t per = kChunkVecs * (16 / elem_bytes(r.dtype));
  return (r.numel + per - 1) / per;
}

// The non-empty tensors in tables of kTensors, and fewer where the chunk count would pass int32.
template <class F>
hipError_t each_table(const moe_tensor_ref* refs, int n, F&& f) {
  TensorTable t;
  t.n = 0, t.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t c = chunks_of(refs[i]);
    if (c == 0) continue;
    if (t.n == kTensors || t.first[t.n] + c > (int64_t(1) << 30)) {
      if (hipError_t err = f(t)) return err;
      t.n = 0, t.first[0] = 0;
    }
    t.in[t.n] = refs[i].data;
    t.out[t.n] = refs[i].out ? refs[i].out : const_cast<void*>(refs[i].data);
    t.numel[t.n] = refs[i].numel;
    t.type[t.n] = static_cast<uint8_t>(refs[i].dtype);
    t.first[t.n + 1] = static_cast<int>(t.first[t.n] + c);
    ++t.n;
  }
  return t.n ? f(t) : hipSuccess;
}

// workgroups of a launch: eight to a compute unit stream at the memory's rate
int grid_of(int chunks) { return std::min(chunks, 8 * device_cu_count()); }

}  // namespace

size_t grad_sumsq_workspace_bytes(const moe_tensor_ref* refs, int n) {
  size_t parts = 0;
  (void)each_table(refs, n, [&](const TensorTable& t) {
    parts += grid_of(t.first[t.n]);
    return hipSuccess;
  });
  return parts * sizeof(double);
}

hipError_t launch_grad_sumsq(const moe_tensor_ref* refs, int n, double* sumsq, void* ws,
                             hipStream_t s) {
  double* part = static_cast<double*>(ws);
  int parts = 0;
  hipError_t err = each_table(refs, n, [&](const TensorTable& t) {
    const int grid = grid_of(t.first[t.n]);
    sumsq_kernel<<<grid, kThreads, 0, s>>>(t, part + parts);
    parts += grid;
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  sumsq_join_kernel<<<1, 1024, 0, s>>>(part, parts, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_tensor_ref* refs, int n, const double* sumsq, float max_norm,
                            float* norm, hipStream_t s) {
  hipError_t err = each_table(refs, n, [&](const TensorTable& t) {
    clip_kernel<<<grid_of(t.first[t.n]), kThreads, 0, s>>>(t, sumsq, max_norm, norm);
    norm = nullptr;
    return hipGetLastError();
  });
  if (err != hipSuccess || !norm) return err;
  TensorTable none;
  none.n = 0, none.first[0] = 0;
  clip_kernel<<<1, kThreads, 0, s>>>(none, sumsq, max_norm, norm);
  return hipGetLastError();
}

bool grad_clip_overlaps(const moe_tensor_ref* refs, int n) {
  struct Range { uintptr_t a, b; bool written; };
  std::vector<Range> r;
  r.reserve(2 * size_t(n));
  for (int i = 0; i < n; ++i) {
    if (refs[i].numel == 0) continue;
    const uintptr_t bytes = uintptr_t(refs[i].numel * elem_bytes(refs[i].dtype));
    const uintptr_t in = reinterpret_cast<uintptr_t>(refs[i].data);
    const uintptr_t out = refs[i].out ? reinterpret_cast<uintptr_t>(refs[i].out) : in;
    r.push_back({out, out + bytes, true});
    if (in != out) r.push_back({in, in + bytes, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
  uintptr_t any = 0, written = 0;
  for (const Range& x : r) {
    if (x.a < (x.written ? any : written)) return true;
    any = std::max(any, x.b);
    if (x.written) written = std::max(written, x.b);
  }
  return false;
}

}  // namespace moe
