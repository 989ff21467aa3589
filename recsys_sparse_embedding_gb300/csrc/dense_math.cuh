// Activations of the dense operators and their derivatives, in fp32.
//   SiLU  z p, p = 1 / (1 + exp(-z));          derivative p (1 + z (1 - p))
//   GELU  z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2; derivative Phi(z) + z phi(z)
// exp and the reciprocal are the hardware's approximations (a few 2^-23
// relative, results below 2^-126 as zero): below the rounding of a bf16 result
// and within a few units of an fp32 one.
#pragma once
#include <cuda_runtime.h>

#include "dinsparse.h"

namespace dsf {

// 1 / (1 + exp(-z)); 0 for z far below zero, 1 far above
__device__ __forceinline__ float sigmoid(float z) {
  float e, p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.f + e));
  return p;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == DSF_ACT_RELU) return z < 0.f ? 0.f : z;  // (a NaN stays)
  if (ACT == DSF_ACT_SILU) return z * sigmoid(z);
  if (ACT == DSF_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
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
    const float cdf = 0.5f * (1.f + erff(z * 0.70710678118654752f));
    return make_float2(z * cdf, fmaf(z, 0.3989422804014327f * __expf(-0.5f * z * z), cdf));
  }
  return make_float2(z, 1.f);
}

}  // namespace dsf
