// Activations of the dense operators and their derivatives, in fp32.
//   SiLU  z p, p = 1 / (1 + exp(-z));          derivative p (1 + z (1 - p))
//   GELU  z Phi(z);                            derivative Phi(z) + z phi(z)
// exp and the reciprocal are the hardware's approximations (a few 2^-23
// relative, results below 2^-126 as zero): below the rounding of a bf16 result
// and within a few units of an fp32 one. Phi is taken as
//   Phi(-|z|) = exp(-z^2 / 2) t P(t), t = 1 / (1 + x / 2), x = |z| / sqrt 2,
// with a polynomial P of degree 8 that was fitted to erfc(x) exp(x^2) / 2 by
// Remez's exchange for the least relative error (0 <= x <= 9.4, where exp ends:
// 1.0 2^-24 with the rounded coefficients). So small values keep their digits:
// Phi is off by at most (1.25 z^2 + 32) 2^-24 of itself, the first part from the
// exponent's roundings, which one rounding of z would cost as well. Its exp(-z^2
// / 2) is also phi's, so value and derivative take two special functions
// together.
#pragma once
#include <cuda_runtime.h>

#include "dinsparse.h"

namespace dsf {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two values at a time: the fp32 pipes take a pair per instruction.
__device__ __forceinline__ float2 pair(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 operator+(float2 a, float2 b) { return __fadd2_rn(a, b); }

// 1 / (1 + exp(-z)); 0 for z far below zero, 1 far above
__device__ __forceinline__ float2 sigmoid(float2 z) {
  const float2 t = z * pair(-kLog2e);
  const float2 d = make_float2(exp2_fast(t.x), exp2_fast(t.y)) + pair(1.f);
  return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

// Phi(z), and exp(-z^2 / 2) in e.
__device__ __forceinline__ float2 normal_cdf(float2 z, float2& e) {
  const float2 x = make_float2(fabsf(z.x), fabsf(z.y)), y = (z * z) * pair(-0.5f * kLog2e);
  e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
  const float2 d = __ffma2_rn(pair(0.35355339059327376f), x, pair(1.f));
  const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
  float2 s = __ffma2_rn(pair(-0.029465685f), t, pair(0.14195053f));
  s = __ffma2_rn(s, t, pair(-0.2428992f));
  s = __ffma2_rn(s, t, pair(0.13822791f));
  s = __ffma2_rn(s, t, pair(-0.0127546815f));
  s = __ffma2_rn(s, t, pair(0.10110574f));
  s = __ffma2_rn(s, t, pair(0.12161241f));
  s = __ffma2_rn(s, t, pair(0.14117926f));
  s = __ffma2_rn(s, t, pair(0.1410437f));
  const float2 half = (s * t) * e, rest = __ffma2_rn(half, pair(-1.f), pair(1.f));
  return make_float2(z.x < 0.f ? half.x : rest.x, z.y < 0.f ? half.y : rest.y);
}

template <int ACT>
__device__ __forceinline__ float2 act_value(float2 z) {
  if (ACT == DSF_ACT_RELU) return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);  // (a NaN stays)
  if (ACT == DSF_ACT_SILU) return z * sigmoid(z);
  if (ACT == DSF_ACT_GELU) {
    float2 e;
    return z * normal_cdf(z, e);
  }
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  return act_value<ACT>(pair(z)).x;
}

// act(z) in value, act'(z) in slope
template <int ACT>
__device__ __forceinline__ void act_both(float2 z, float2& value, float2& slope) {
  value = z;
  slope = pair(1.f);
  if (ACT == DSF_ACT_RELU) {
    value = act_value<ACT>(z);
    slope = make_float2(z.x > 0.f ? 1.f : (z.x != z.x ? z.x : 0.f), z.y > 0.f ? 1.f : (z.y != z.y ? z.y : 0.f));
  }
  if (ACT == DSF_ACT_SILU) {
    const float2 p = sigmoid(z);
    value = z * p;
    slope = p * __ffma2_rn(z, __ffma2_rn(p, pair(-1.f), pair(1.f)), pair(1.f));
  }
  if (ACT == DSF_ACT_GELU) {
    float2 e;
    const float2 cdf = normal_cdf(z, e);
    value = z * cdf;
    slope = __ffma2_rn(z * pair(0.3989422804014327f), e, cdf);
  }
}

}  // namespace dsf
