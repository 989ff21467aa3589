// Column sums of a [rows, N] fp32 matrix of partial sums, in a fixed order:
// the last step of the bias and norm-weight gradients.
#pragma once
#include <cuda_runtime.h>

#include "pdl.cuh"

namespace dsf {

// out[n] = sum over r of P[r][n]. A block takes 8 columns (32-byte sectors):
// lane l of warp g adds rows 4 g + l / 8, + 128, ... of column l % 8 in order
// (four loads in flight), then the 128 sums are added in a fixed tree, so the
// result does not depend on timing. (Latency is what counts here: 608 x 256 took
// 19 us with 32 columns and 8 warps to a block, 7 with 32 columns and 32 warps.)
template <int = 0>  // (a template so that several units may include it)
__global__ void __launch_bounds__(1024) colsum_kernel(const float* __restrict__ P, long long rows, int N,
                                                      float* __restrict__ out) {
  constexpr int W = 32, U = 4, R = 4 * W;
  __shared__ float part[W][8];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = lane & 7;
  const int n = blockIdx.x * 8 + c;
  pdl_go();
  pdl_wait();
  float s = 0.f;
  if (n < N) {
    for (long long r0 = 4 * g + (lane >> 3); r0 < rows; r0 += R * U) {
      float v[U];
#pragma unroll
      for (int t = 0; t < U; ++t) v[t] = r0 + R * t < rows ? P[(r0 + R * t) * N + n] : 0.f;
#pragma unroll
      for (int t = 0; t < U; ++t) s += v[t];
    }
  }
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if (lane < 8) part[g][c] = s;
  __syncthreads();
  if (g == 0) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < W / 4; ++k) s += part[(lane >> 3) * (W / 4) + k][c];
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (lane < 8 && n < N) out[n] = s;
  }
}

// The same for wide matrices: a block takes 32 columns, lane l of warp g rows
// g, g + 32, ... of column l (eight loads in flight). (300 x 8192: 20 us by
// blocks of 8 columns, which are then many and short.)
template <int = 0>
__global__ void __launch_bounds__(1024) colsum_wide_kernel(const float* __restrict__ P, long long rows, int N,
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
  // warp g adds column g: its 32 sums by a fixed tree
  float v = part[lane][g];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blockIdx.x * 32 + g < N) out[blockIdx.x * 32 + g] = v;
}

inline bool colsum(const float* P, long long rows, int N, float* out, cudaStream_t s) {
  if (N >= 2048) return pdl_launch(colsum_wide_kernel<>, dim3(unsigned((N + 31) / 32)), 1024, s, P, rows, N, out);
  return pdl_launch(colsum_kernel<>, dim3(unsigned((N + 7) / 8)), 1024, s, P, rows, N, out);
}

}  // namespace dsf
