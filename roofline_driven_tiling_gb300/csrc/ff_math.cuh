// ff_math.cuh -- conversions and activation functions of the feed-forward operators, in FP32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "ff_internal.h"

namespace t2s {
namespace ff {

template <int KIND>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (KIND == kBf16) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  } else {
    return __half2float(__ushort_as_half(v));
  }
}

// The two values of a 32-bit word, low half first.
template <int KIND>
__device__ __forceinline__ float2 to_f32x2(uint32_t v) {
  if constexpr (KIND == kBf16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

// Rounded to nearest even, `lo` in the low half.
template <int KIND>
__device__ __forceinline__ uint32_t pack_f32(float lo, float hi) {
  if constexpr (KIND == kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int KIND>
__device__ __forceinline__ uint16_t from_f32(float v) {
  if constexpr (KIND == kBf16) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  } else {
    return __half_as_ushort(__float2half_rn(v));
  }
}

constexpr float kGeluC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 2^x and 1 / x by the hardware's approximations (2 and 1 ulp; results under 2^-126 become 0). The
// epilogues' arithmetic is bound by instructions, and these are one each.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2E = 1.4426950408889634f;

// The logistic function of v from w = -v log2(e): 2^w overflowing to infinity gives the limit 0.
__device__ __forceinline__ float logistic_of(float w) { return reciprocal_approx(1.0f + exp2_approx(w)); }

// P(-|x|), the normal distribution's tail, = erfc(|x| / sqrt 2) / 2 by Abramowitz and Stegun's formula
// 7.1.26 (a polynomial of degree 5 in 1 / (1 + p |x| / sqrt 2) times e^(-x^2 / 2), off by at most
// 7.5e-8 in P). erff in its place made the epilogue of 2048^3 with gelu the longer half of the kernel.
// `e` is e^(-x^2 / 2).
__device__ __forceinline__ float normal_tail(float x, float e) {
  const float t = reciprocal_approx(fmaf(0.3275911f * 0.70710678118654752f, fabsf(x), 1.0f));
  float q = 0.5f * 1.061405429f;
  q = fmaf(q, t, 0.5f * -1.453152027f);
  q = fmaf(q, t, 0.5f * 1.421413741f);
  q = fmaf(q, t, 0.5f * -0.284496736f);
  q = fmaf(q, t, 0.5f * 0.254829592f);
  return q * t * e;
}

// act(z): relu max(z, 0) (a NaN passes), silu z s(z), gelu z P(z) = z (1 + erf(z / sqrt 2)) / 2,
// gelu_tanh z (1 + tanh u) / 2 = z s(2 u) with u = c (z + a z^3).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == T2S_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == T2S_ACT_SILU) return z * logistic_of(-kLog2E * z);
  if constexpr (ACT == T2S_ACT_GELU) {
    const float q = normal_tail(z, exp2_approx((-0.5f * kLog2E) * z * z));
    return z * (z > 0.0f ? 1.0f - q : q);
  }
  if constexpr (ACT == T2S_ACT_GELU_TANH)
    return z * logistic_of(z * fmaf(-2.0f * kLog2E * kGeluC * kGeluA, z * z, -2.0f * kLog2E * kGeluC));
  return z;
}

// z within [-100, 100]; a NaN stays.
__device__ __forceinline__ float within_100(float z) {
  float x;
  asm("max.NaN.f32 %0, %1, 0fC2C80000;\n\tmin.NaN.f32 %0, %0, 0f42C80000;" : "=f"(x) : "f"(z));
  return x;
}

// Both act(z) and act'(z) from one exponential. From |z| = 100 on every slope here is exactly 0 or 1
// in FP32 (e^100 overflows), so slopes take z clamped there: no product is 0 times infinity.
template <int ACT>
__device__ __forceinline__ void act_value_slope(float z, float& value, float& slope) {
  if constexpr (ACT == T2S_ACT_NONE) {
    value = z;
    slope = 1.0f;
  } else if constexpr (ACT == T2S_ACT_RELU) {
    value = z < 0.0f ? 0.0f : z;
    slope = z <= 0.0f ? 0.0f : 1.0f;
  } else {
    const float x = within_100(z), x2 = x * x;
    if constexpr (ACT == T2S_ACT_SILU) {
      // s + x s (1 - s)
      const float s = logistic_of(-kLog2E * x);
      slope = fmaf(x, fmaf(-s, s, s), s);
      value = z * s;
    } else if constexpr (ACT == T2S_ACT_GELU) {
      // P(x) + x p(x) with the normal distribution P and its density p.
      const float e = exp2_approx((-0.5f * kLog2E) * x2), q = normal_tail(x, e);
      const float d = x > 0.0f ? 1.0f - q : q;
      slope = fmaf(0.39894228040143268f * x, e, d);
      value = z * d;
    } else {
      // s + x s (1 - s) v' with v = 2 c (x + a x^3)
      const float s = logistic_of(x * fmaf(-2.0f * kLog2E * kGeluC * kGeluA, x2, -2.0f * kLog2E * kGeluC));
      slope = fmaf(x * fmaf(-s, s, s), fmaf(6.0f * kGeluC * kGeluA, x2, 2.0f * kGeluC), s);
      value = z * s;
    }
  }
}

// Calls f with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case T2S_ACT_RELU: f(std::integral_constant<int, T2S_ACT_RELU>{}); break;
    case T2S_ACT_SILU: f(std::integral_constant<int, T2S_ACT_SILU>{}); break;
    case T2S_ACT_GELU: f(std::integral_constant<int, T2S_ACT_GELU>{}); break;
    case T2S_ACT_GELU_TANH: f(std::integral_constant<int, T2S_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, T2S_ACT_NONE>{}); break;
  }
}

}  // namespace ff
}  // namespace t2s
