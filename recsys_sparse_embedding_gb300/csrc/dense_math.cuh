// Activations of the dense operators and their derivatives, in fp32.
//   SiLU  z p, p = 1 / (1 + exp(-z));          derivative p (1 + z (1 - p))
//   GELU  z Phi(z);                            derivative Phi(z) + z phi(z)
// exp and the reciprocal are the hardware's approximations (a few 2^-23
// relative, results below 2^-126 as zero): below the rounding of a bf16 result
// and within a few units of an fp32 one. Phi is taken from the rational form
// 7.1.26 of Abramowitz and Stegun's Handbook of Mathematical Functions,
//   erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + p x), x >= 0,
// within 1.5e-7, with x = |z| / sqrt 2: its exp(-z^2 / 2) is also phi's, so
// value and derivative take two special functions together.
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

// 1 / (1 + exp(-z)); 0 for z far below zero, 1 far above
__device__ __forceinline__ float sigmoid(float z) { return rcp_fast(1.f + exp2_fast(-kLog2e * z)); }

// Phi(z), and exp(-z^2 / 2) in e. Below zero Phi is half of erfc itself.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  e = exp2_fast(-kLog2e * (x * x));
  const float t = rcp_fast(fmaf(0.3275911f, x, 1.f));
  float s = fmaf(1.061405429f, t, -1.453152027f);
  s = fmaf(s, t, 1.421413741f);
  s = fmaf(s, t, -0.284496736f);
  s = fmaf(s, t, 0.254829592f);
  const float half = 0.5f * s * t * e;
  return z < 0.f ? half : 1.f - half;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == DSF_ACT_RELU) return z < 0.f ? 0.f : z;  // (a NaN stays)
  if (ACT == DSF_ACT_SILU) return z * sigmoid(z);
  if (ACT == DSF_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  return z;
}

// act(z) and act'(z) together
template <int ACT>
__device__ __forceinline__ float2 act_both(float z) {
  if (ACT == DSF_ACT_RELU) return z > 0.f ? make_float2(z, 1.f) : make_float2(z < 0.f ? 0.f : z, z != z ? z : 0.f);
  if (ACT == DSF_ACT_SILU) {
    const float p = sigmoid(z);
    return make_float2(z * p, p * fmaf(z, 1.f - p, 1.f));
  }
  if (ACT == DSF_ACT_GELU) {
    float e;
    const float cdf = normal_cdf(z, e);
    return make_float2(z * cdf, fmaf(z, 0.3989422804014327f * e, cdf));
  }
  return make_float2(z, 1.f);
}

}  // namespace dsf
