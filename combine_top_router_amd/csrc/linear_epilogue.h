// What the dense products' epilogues share: bias, activation, residual, the
// pre-activation kept for the backward, and the outputs' types.
#pragma once

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {
namespace {

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

// e^x and 1/x by the hardware's base-2 exponential and reciprocal: within
// 2^-22 (|x| + 2) of e^x, far inside what a 16-bit or summed fp32 value shows.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}

// The normal distribution function, by Hastings' form of the error function
// (Abramowitz and Stegun 7.1.23-28), erfc(x) = t P(t) e^(-x^2), t = 1 / (1 + p x),
// x >= 0, with eight terms fitted here to the relative error (1.1e-7 up to x = 10;
// the book's five terms are within 1.5e-7 absolute, 0.16 % off at z = -5 and 2 % at -10).
// With the hardware's exponential within 2^-21 (1 + z^2 / 2) of itself: about what half a
// step of z does to it. The library's erfcf took a third of the time of a
// 1023x4096x14336 product with gelu. g receives e^(-z^2/2).
__device__ __forceinline__ float normal_cdf(float z, float& g) {
  constexpr float kP[8] = {0.24252208f, 0.24425802f, 0.20570278f, 0.24429801f,
                           -0.08078131f, 0.37818462f, -0.30707936f, 0.07289512f};
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(1.f + 0.43f * x);
  g = __expf(-x * x);
  float poly = kP[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) poly = kP[i] + t * poly;
  const float half = 0.5f * g * t * poly;
  return z < 0.f ? half : 1.f - half;
}

__device__ __forceinline__ float act_of(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z != z ? z : fmaxf(z, 0.f);  // NaN stays NaN
    case MOE_ACT_SILU: return z * sigmoid(z);
    case MOE_ACT_GELU: {
      float g;
      return z * normal_cdf(z, g);
    }
    default: return z;
  }
}

// (an infinite z, as fp16 stores what is past its range: clamped where the slopes
// are 0 and 1 already, or z times a vanishing factor would be NaN; NaN stays NaN)
__device__ __forceinline__ float act_slope(float z, int act) {
  z = z != z ? z : fminf(fmaxf(z, -1e4f), 1e4f);
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACT_GELU: {
      float g;
      const float c = normal_cdf(z, g);
      return c + z * g * 0.39894228040143268f;
    }
    default: return 1.f;
  }
}

__device__ __forceinline__ u32x4 load8x16(const uint16_t* p) {
  return *reinterpret_cast<const u32x4*>(p);
}

template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
  switch (act) {  // one uniform branch for all of them
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_of(v[i], MOE_ACT_RELU);
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_of(v[i], MOE_ACT_SILU);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_of(v[i], MOE_ACT_GELU);
      break;
    default: break;
  }
}

// Where a block of outputs begins: offsets inside it fit 32 bits.
struct Block {
  char* out;
  const uint16_t* res;
  uint16_t* pre;
  int ldo, ldr, ldp;
  __device__ __forceinline__ Block(const Epilogue& e, int64_t m, int64_t n)
      : out(static_cast<char*>(e.out) + (m * e.ldo + n) * (e.out_f32 ? 4 : 2)),
        res(e.res ? e.res + m * e.ldr + n : nullptr), pre(e.pre ? e.pre + m * e.ldp + n : nullptr),
        ldo(int(e.ldo)), ldr(int(e.ldr)), ldp(int(e.ldp)) {}
};

// Columns c .. c+7 of a block's row r from their sums v, the columns' bias and
// the residual's values: rows that start 16-byte aligned.
__device__ __forceinline__ void finish8(const Epilogue& e, const Block& b, int r, int c,
                                        float (&v)[8], const float (&bias)[8], const u32x4& res) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += bias[i];
  if (e.pre) *reinterpret_cast<u32x4*>(b.pre + (r * b.ldp + c)) = pack8x16(v, e.f16);
  act_all(v, e.act);
  if (e.res) {
    float x[8];
    unpack8x16(res, x, e.f16);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
  }
  if (e.out_f32) {
    float* o = reinterpret_cast<float*>(b.out) + (r * b.ldo + c);
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(o));
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(o + 4));
  } else {
    __builtin_nontemporal_store(
        pack8x16(v, e.f16),
        reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(b.out) + (r * b.ldo + c)));
  }
}

// Column c of the rows r, r + step, ... of a block, from their sums v, as far as
// they lie before `end`: rows of any alignment.
template <int N>
__device__ __forceinline__ void finish_column(const Epilogue& e, const Block& b, int r, int step,
                                              int end, int c, float (&v)[N], float bias) {
  uint16_t x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = e.res && r + i * step < end ? b.res[(r + i * step) * b.ldr + c] : 0;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += bias;
  if (e.pre) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (r + i * step < end) b.pre[(r + i * step) * b.ldp + c] = to16(v[i], e.f16);
  }
  act_all(v, e.act);
  if (e.res) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += from16(x[i], e.f16);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (r + i * step >= end) continue;
    if (e.out_f32) reinterpret_cast<float*>(b.out)[(r + i * step) * b.ldo + c] = v[i];
    else reinterpret_cast<uint16_t*>(b.out)[(r + i * step) * b.ldo + c] = to16(v[i], e.f16);
  }
}

}  // namespace
}  // namespace moe
