// Activations of the dense operators and their derivatives, in fp32.
//   SiLU  z p, p = 1 / (1 + exp(-z));          derivative p (1 + z (1 - p))
//   GELU  z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2; derivative Phi(z) + z phi(z)
// exp and the quotient are the fast forms: about 2^-21 relative, below the
// rounding of a bf16 result and within a few units of an fp32 one.
#pragma once
#include <cuda_runtime.h>

#include "dinsparse.h"

namespace dsf {

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == DSF_ACT_RELU) return z < 0.f ? 0.f : z;  // (a NaN stays)
  if (ACT == DSF_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if (ACT == DSF_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  return z;
}

// act(z) and act'(z) together
template <int ACT>
__device__ __forceinline__ float2 act_both(float z) {
  if (ACT == DSF_ACT_RELU) return z > 0.f ? make_float2(z, 1.f) : make_float2(z < 0.f ? 0.f : z, z != z ? z : 0.f);
  if (ACT == DSF_ACT_SILU) {
    const float p = __fdividef(1.f, 1.f + __expf(-z));
    return make_float2(z * p, p * fmaf(z, 1.f - p, 1.f));
  }
  if (ACT == DSF_ACT_GELU) {
    const float cdf = 0.5f * (1.f + erff(z * 0.70710678118654752f));
    return make_float2(z * cdf, fmaf(z, 0.3989422804014327f * __expf(-0.5f * z * z), cdf));
  }
  return make_float2(z, 1.f);
}

}  // namespace dsf
