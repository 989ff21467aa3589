// Column sums of a [rows, N] fp32 matrix of partial sums, in a fixed order:
// the last step of the bias and norm-weight gradients.
#pragma once
#include <cuda_runtime.h>

namespace dsf {

// out[n] = sum over r of P[r][n]. A block of 8 warps takes 32 columns: warp g
// adds rows g, g + 8, g + 16, ... in order (four loads in flight), then warp 0
// adds the eight sums in warp order, so the result does not depend on timing.
// (One per unit that includes it; a template so that the units may share it.)
template <int = 0>
__global__ void __launch_bounds__(256) colsum_kernel(const float* __restrict__ P, long long rows, int N,
                                                     float* __restrict__ out) {
  __shared__ float part[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (n < N) {
    for (long long r0 = g; r0 < rows; r0 += 32) {
      float v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = r0 + 8 * t < rows ? P[(r0 + 8 * t) * N + n] : 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) s += v[t];
    }
  }
  part[g][lane] = s;
  __syncthreads();
  if (g == 0 && n < N) {
    float r = part[0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k) r += part[k][lane];
    out[n] = r;
  }
}

inline bool colsum(const float* P, long long rows, int N, float* out, cudaStream_t s) {
  colsum_kernel<><<<unsigned((N + 31) / 32), 256, 0, s>>>(P, rows, N, out);
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace dsf
