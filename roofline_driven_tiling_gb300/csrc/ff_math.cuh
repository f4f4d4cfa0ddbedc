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

// Two FP32 values in a 64-bit register, for the packed instructions: half the issue slots of the
// epilogues' additions, products and polynomials.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t exp2_of(uint64_t v) {
  const float2 x = halves(v);
  return pack2(exp2_approx(x.x), exp2_approx(x.y));
}
__device__ __forceinline__ uint64_t reciprocal_of(uint64_t v) {
  const float2 x = halves(v);
  return pack2(reciprocal_approx(x.x), reciprocal_approx(x.y));
}
// max(x, 0); a NaN stays.
__device__ __forceinline__ uint64_t positive_of(uint64_t v) {
  float2 x = halves(v);
  asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(x.x));
  asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(x.y));
  return pack2(x.x, x.y);
}

// -P(-|x|) e^(x^2 / 2), the normal distribution's tail over its exponential, for 0 <= ax = |x|: a polynomial in
// t = 1 / (1 + p |x|), of degree 6 with p = 0.3, whose greatest relative error over 0 <= |x| <= 14 is least
// (1.9e-6 = 2^-19; a fit by least squares, reweighted until its extremes are level). Relative, because for negative
// z the tail is gelu(z) itself, which 16-bit types hold down to -12; with the exponential's own rounding gelu is
// within 2^-16 of it there. Negative, so that gelu is max(z, 0) plus a product. erff in its place made the epilogue
// of 2048^3 with gelu the longer half of the kernel.
__device__ __forceinline__ uint64_t minus_scaled_tail(uint64_t ax) {
  const uint64_t t = reciprocal_of(fma2(ax, both(0.3f), both(1.0f)));
  uint64_t q = fma2(both(0.0845932673f), t, both(-0.240572934f));
  q = fma2(q, t, both(0.0486446416f));
  q = fma2(q, t, both(-0.16476465f));
  q = fma2(q, t, both(-0.106704458f));
  q = fma2(q, t, both(-0.121274716f));
  q = fma2(q, t, both(7.97905242e-05f));
  return q;
}

// act(z) of two values: relu max(z, 0), silu z s(z), gelu z P(z) = z (1 + erf(z / sqrt 2)) / 2 =
// max(z, 0) - |z| P(-|z|), gelu_tanh z (1 + tanh u) / 2 = z s(2 u) with u = c (z + a z^3). A NaN stays.
template <int ACT>
__device__ __forceinline__ uint64_t act_pair(uint64_t z) {
  if constexpr (ACT == T2S_ACT_RELU) return positive_of(z);
  if constexpr (ACT == T2S_ACT_SILU)
    return mul2(z, reciprocal_of(add2(exp2_of(mul2(z, both(-kLog2E))), both(1.0f))));
  if constexpr (ACT == T2S_ACT_GELU) {
    // Beyond 100 the tail is 0, and |z| need not grow to meet it.
    const float2 x = halves(z);
    const uint64_t ax = pack2(fminf(fabsf(x.x), 100.0f), fminf(fabsf(x.y), 100.0f));
    return fma2(ax, mul2(minus_scaled_tail(ax), exp2_of(mul2(mul2(ax, ax), both(-0.5f * kLog2E)))), positive_of(z));
  }
  if constexpr (ACT == T2S_ACT_GELU_TANH) {
    const uint64_t w = mul2(z, fma2(mul2(z, z), both(-2.0f * kLog2E * kGeluC * kGeluA), both(-2.0f * kLog2E * kGeluC)));
    return mul2(z, reciprocal_of(add2(exp2_of(w), both(1.0f))));
  }
  return z;
}

// max(z, -100), min(z, 100) and min(|z|, 100); a NaN stays.
__device__ __forceinline__ float least_100(float z) {
  float x;
  asm("max.NaN.f32 %0, %1, 0fC2C80000;" : "=f"(x) : "f"(z));
  return x;
}
__device__ __forceinline__ float most_100(float z) {
  float x;
  asm("min.NaN.f32 %0, %1, 0f42C80000;" : "=f"(x) : "f"(z));
  return x;
}
__device__ __forceinline__ float magnitude_100(float z) { return most_100(fabsf(z)); }

// Both act(z) and act'(z) of two values, from one exponential each. From |z| = 100 on every slope
// here is exactly 0 or 1 in FP32 (e^100 overflows), so slopes take z clamped there, and values take it
// clamped below (binary16 keeps a gate of -70000 as -inf): no product is 0 times infinity.
template <int ACT>
__device__ __forceinline__ void act_pair_slope(uint64_t z, uint64_t& value, uint64_t& slope) {
  const float2 f = halves(z);
  if constexpr (ACT == T2S_ACT_NONE) {
    value = z;
    slope = both(1.0f);
  } else if constexpr (ACT == T2S_ACT_RELU) {
    value = positive_of(z);
    slope = pack2(f.x <= 0.0f ? 0.0f : 1.0f, f.y <= 0.0f ? 0.0f : 1.0f);
  } else if constexpr (ACT == T2S_ACT_GELU) {
    // P(z) + z p(z) with the normal distribution P and its density p: with r = P(-|z|) - |z| p(z) it is r for
    // negative z and 1 - r for the others.
    const uint64_t ax = pack2(magnitude_100(f.x), magnitude_100(f.y));
    const uint64_t e = exp2_of(mul2(mul2(ax, ax), both(-0.5f * kLog2E))), q = minus_scaled_tail(ax);
    const uint64_t minus_r = mul2(fma2(ax, both(0.39894228040143268f), q), e);
    const float2 r = halves(minus_r);
    slope = pack2(f.x > 0.0f ? r.x + 1.0f : -r.x, f.y > 0.0f ? r.y + 1.0f : -r.y);
    value = fma2(ax, mul2(q, e), positive_of(z));
  } else {
    // s(v) + x s (1 - s) v' with v = x (silu) or 2 c (x + a x^3) (gelu_tanh)
    constexpr bool kSilu = ACT == T2S_ACT_SILU;
    const float2 low = make_float2(least_100(f.x), least_100(f.y));
    const uint64_t x = pack2(most_100(low.x), most_100(low.y)), x2 = mul2(x, x);
    const uint64_t w = kSilu ? mul2(x, both(-kLog2E))
                             : mul2(x, fma2(x2, both(-2.0f * kLog2E * kGeluC * kGeluA), both(-2.0f * kLog2E * kGeluC)));
    const uint64_t s = reciprocal_of(add2(exp2_of(w), both(1.0f)));
    const uint64_t bell = fma2(mul2(s, both(-1.0f)), s, s);
    slope = kSilu ? fma2(x, bell, s)
                  : fma2(mul2(x, bell), fma2(x2, both(6.0f * kGeluC * kGeluA), both(2.0f * kGeluC)), s);
    value = mul2(pack2(low.x, low.y), s);
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
