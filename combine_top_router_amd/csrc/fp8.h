// Values in 8 bits: e4m3 with an fp32 scale for a run of 128.
//
//   s = max(amax / 448, 2^-126),  q = e4m3(v * (1 / s))
//
// amax: the largest magnitude among the run's finite values; 448 is e4m3's
// largest value, so that nothing saturates. A value that is not finite is
// stored as NaN (e4m3 has no infinity) and leaves the others as they are.
// Quotient, reciprocal, product: fp32, each rounded once; then one rounding to
// e4m3, half a step of which is 2^-4 of the value (2^-10 s near 0).
#pragma once

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kRun = 128;  // values that share a scale

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false);
}

// Over each 16 lanes, the result in all of them: exchanges within quads, then
// mirrored halves and rows.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, dpp<0xb1>(v));
  v = max(v, dpp<0x4e>(v));
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}
__device__ __forceinline__ float sum16(float v) {
  auto other = [](float x, auto ctrl) {
    return __uint_as_float(dpp<decltype(ctrl)::value>(__float_as_uint(x)));
  };
  v += other(v, std::integral_constant<int, 0xb1>{});
  v += other(v, std::integral_constant<int, 0x4e>{});
  v += other(v, std::integral_constant<int, 0x141>{});
  return v + other(v, std::integral_constant<int, 0x140>{});
}

// |v| as an integer that orders like it; 0 where v is not finite.
__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

template <int N>
__device__ __forceinline__ uint32_t magnitude(const float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, magnitude(v[i]));
  return m;
}

__device__ __forceinline__ float scale_of(uint32_t amax) {
  return fmaxf(__uint_as_float(amax) / 448.f, 0x1p-126f);
}

// Eight values in units of 1 / r, as e4m3.
__device__ __forceinline__ uint2 to_fp8x8(const float (&v)[8], float r) {
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = fabsf(v[i]) < INFINITY ? v[i] * r : NAN;
  uint2 q;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
  q.x = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], w, true);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(u[4], u[5], 0, false);
  q.y = __builtin_amdgcn_cvt_pk_fp8_f32(u[6], u[7], w, true);
  return q;
}

// ---- rows of bf16, fp16 or fp32, eight values at a time (MOE_ROWS_*)

typedef _Float16 f16v2 __attribute__((ext_vector_type(2)));

template <int T>
struct Raw {  // eight values as they lie in memory
  u32x4 v[T == 2 ? 2 : 1];
};

template <int T>
constexpr int elem_bytes() { return T == 2 ? 4 : 2; }

template <int T>
__device__ __forceinline__ Raw<T> load8(const void* p, int64_t at) {
  const u32x4* a = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + at * elem_bytes<T>());
  Raw<T> r;
  r.v[0] = a[0];
  if constexpr (T == 2) r.v[1] = a[1];
  return r;
}

template <int T>
__device__ __forceinline__ void values8(const Raw<T>& r, float (&f)[8]) {
  if constexpr (T == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.v[i / 4][i % 4]);
  } else if constexpr (T == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = r.v[0][i];  // (a bit cast of a vector's element itself takes the first one)
      const f16v2 h = __builtin_bit_cast(f16v2, w);
      f[2 * i] = static_cast<float>(h[0]), f[2 * i + 1] = static_cast<float>(h[1]);
    }
  } else {
    unpack8(r.v[0], f);
  }
}

template <int T>
__device__ __forceinline__ Raw<T> raw8(const float (&f)[8]) {
  Raw<T> r;
  if constexpr (T == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i / 4][i % 4] = __float_as_uint(f[i]);
  } else if constexpr (T == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16v2 h;
      h[0] = static_cast<_Float16>(f[2 * i]), h[1] = static_cast<_Float16>(f[2 * i + 1]);
      r.v[0][i] = __builtin_bit_cast(uint32_t, h);
    }
  } else {
    r.v[0] = pack8(f);
  }
  return r;
}

template <int T>
__device__ __forceinline__ void store8(void* p, int64_t at, const Raw<T>& r) {
  u32x4* a = reinterpret_cast<u32x4*>(static_cast<char*>(p) + at * elem_bytes<T>());
  __builtin_nontemporal_store(r.v[0], a);
  if constexpr (T == 2) __builtin_nontemporal_store(r.v[1], a + 1);
}

__device__ __forceinline__ void store_fp8x8(void* p, int64_t at, const uint2& q) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(u32x2{q.x, q.y},
                              reinterpret_cast<u32x2*>(static_cast<char*>(p) + at));
}

}  // namespace
}  // namespace moe
