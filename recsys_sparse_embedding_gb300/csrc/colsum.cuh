// Column sums of a [rows, N] fp32 matrix of partial sums, in a fixed order:
// the last step of the bias and norm-weight gradients.
#pragma once
#include <cuda_runtime.h>

#include "pdl.cuh"

namespace dsf {

// out[n] = sum over r of P[r][n]. A block of 32 warps takes 32 columns: warp g
// adds rows g, g + 32, g + 64, ... in order (eight loads in flight), then warp
// 0 adds the 32 sums in warp order, so the result does not depend on timing.
// (Latency is what counts here: 608 x 256 took 19 us with 8 warps and four
// loads in flight, the rows in sequence.)
template <int = 0>  // (a template so that several units may include it)
__global__ void __launch_bounds__(1024) colsum_kernel(const float* __restrict__ P, long long rows, int N,
                                                      float* __restrict__ out) {
  constexpr int W = 32, U = 8;
  __shared__ float part[W][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + lane;
  pdl_go();
  pdl_wait();
  float s = 0.f;
  if (n < N) {
    for (long long r0 = g; r0 < rows; r0 += W * U) {
      float v[U];
#pragma unroll
      for (int t = 0; t < U; ++t) v[t] = r0 + W * t < rows ? P[(r0 + W * t) * N + n] : 0.f;
#pragma unroll
      for (int t = 0; t < U; ++t) s += v[t];
    }
  }
  part[g][lane] = s;
  __syncthreads();
  if (g == 0 && n < N) {
    float r = part[0][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) r += part[k][lane];
    out[n] = r;
  }
}

inline bool colsum(const float* P, long long rows, int N, float* out, cudaStream_t s) {
  return pdl_launch(colsum_kernel<>, dim3(unsigned((N + 31) / 32)), 1024, s, P, rows, N, out);
}

}  // namespace dsf
