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

// z s(v) with the logistic s, as a quotient: e^-v overflowing to infinity gives the limit 0.
__device__ __forceinline__ float times_logistic(float z, float v) {
  return __fdividef(z, 1.0f + __expf(-v));
}

// act(z): relu max(z, 0) (a NaN passes), silu z s(z), gelu z (1 + erf(z / sqrt 2)) / 2,
// gelu_tanh z (1 + tanh u) / 2 = z s(2 u) with u = c (z + a z^3).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == T2S_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == T2S_ACT_SILU) return times_logistic(z, z);
  if constexpr (ACT == T2S_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  if constexpr (ACT == T2S_ACT_GELU_TANH)
    return times_logistic(z, (2.0f * kGeluC) * (z + kGeluA * z * z * z));
  return z;
}

// Both act(z) and act'(z). From |z| = 100 on every slope here is exactly 0 or 1 in FP32 (e^100
// overflows), so z is clamped there before products that would be 0 times infinity.
template <int ACT>
__device__ __forceinline__ void act_value_slope(float z, float& value, float& slope) {
  if constexpr (ACT == T2S_ACT_NONE) {
    value = z;
    slope = 1.0f;
  } else if constexpr (ACT == T2S_ACT_RELU) {
    value = z < 0.0f ? 0.0f : z;
    slope = z <= 0.0f ? 0.0f : 1.0f;
  } else {
    value = act_value<ACT>(z);
    const float x = z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z;  // a NaN stays
    if constexpr (ACT == T2S_ACT_SILU) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-x));
      slope = s * (1.0f + x * (1.0f - s));
    } else if constexpr (ACT == T2S_ACT_GELU) {
      // P(x) + x p(x) with the normal distribution P and its density p.
      slope = 0.5f * (1.0f + erff(x * 0.70710678118654752f)) +
              x * (0.39894228040143268f * __expf(-0.5f * x * x));
    } else {
      const float u2 = (2.0f * kGeluC) * (x + kGeluA * x * x * x);
      const float s = __fdividef(1.0f, 1.0f + __expf(-u2));
      slope = s + x * s * (1.0f - s) * (2.0f * kGeluC) * (1.0f + 3.0f * kGeluA * x * x);
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
