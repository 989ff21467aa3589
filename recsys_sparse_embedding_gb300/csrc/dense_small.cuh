// Forward of a few rows, or of small layers: the weights straight from memory,
// on the CUDA cores.
//
// y[m][n] = sum over k of x[m][k] W[n][k] needs 2 M operations per weight, so
// up to a handful of rows the weights' bytes are all that counts: a tensor-core
// tile would use 8 of its 128 rows. A warp takes one output column (a gated
// layer: its gate and up rows), its lanes side by side along K in 16-byte
// vectors, several in flight; x (a few KB) stays in L1. More than 8 rows go by
// eights. fp32 sums, then
// the operator's epilogue in the lane of each row.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dense_math.cuh"
#include "pdl.cuh"

namespace dsf {
namespace dense {

constexpr int kSmallM = 8;

struct SmallArgs {
  const void *x, *W;
  long long ldx, ldw;
  const float *bias, *xs, *ws;
  const void* res;
  long long ldr;
  void* y;
  long long ldy;
  int M, N, K, act;
  int col_blocks;  // blocks per 8 rows (set by the launch)
};

__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case DSF_ACT_RELU: return act_value<DSF_ACT_RELU>(z);
    case DSF_ACT_SILU: return act_value<DSF_ACT_SILU>(z);
    case DSF_ACT_GELU: return act_value<DSF_ACT_GELU>(z);
    default: return z;
  }
}

__device__ __forceinline__ float elem(float v) { return v; }
__device__ __forceinline__ float elem(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem(__nv_fp8_e4m3 v) { return float(v); }

// the elements of a 16-byte vector
__device__ __forceinline__ void unpack(const uint4& u, float* v, float) {
  v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float* v, __nv_bfloat16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float* v, __nv_fp8_e4m3) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[i] >> (16 * h)), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      v[4 * i + 2 * h] = f.x;
      v[4 * i + 2 * h + 1] = f.y;
    }
}

// NC: output columns per warp; x is read, and unpacked to fp32, once for all
// of them. Loads are unconditional in the row index (rows past the last repeat
// it), so that all of a step's are in flight together: with a loop that stopped
// at the last row, 8 x 1024 -> 4096 took 12 us instead of 6.5.
template <class T, class TO, int MT, int NC, bool GATED, bool VEC, bool ONE>
__global__ void __launch_bounds__(256) small_kernel(const SmallArgs a) {
  constexpr int NB = GATED ? 2 : 1, R = NB * NC;  // weight rows per warp: the columns, then their up rows
  constexpr int E = VEC ? 16 / int(sizeof(T)) : 1;
  // vectors (or elements) of each row per lane and step (ONE: a row is one step of 32 lanes)
  constexpr int U = VEC ? (ONE ? 1 : (R >= 4 ? 2 : 4)) : 4;
  const int chunk = int(blockIdx.x) / a.col_blocks, n_blk = int(blockIdx.x) - chunk * a.col_blocks;
  const int lane = threadIdx.x & 31, n0 = (n_blk * 8 + int(threadIdx.x >> 5)) * NC;
  pdl_go();
  pdl_wait();
  if (n0 >= a.N) return;
  const int m0 = chunk * MT, rows = min(MT, a.M - m0);
  const T* x[MT];  // (rows past the last read the last one)
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = static_cast<const T*>(a.x) + (long long)(m0 + min(m, rows - 1)) * a.ldx;
  const T* w[R];
#pragma unroll
  for (int c = 0; c < R; ++c)  // (columns past the last read the last one's weights)
    w[c] = static_cast<const T*>(a.W) + (long long)(min(n0 + c % NC, a.N - 1) + (c / NC) * a.N) * a.ldw;
  float acc[R][MT];
#pragma unroll
  for (int c = 0; c < R; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[c][m] = 0.f;
  const int nv = a.K / E;  // (VEC: K is a whole number of vectors)
  for (int v0 = lane; v0 < nv; v0 += 32 * U) {
    if constexpr (VEC) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 b[R][U];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int c = 0; c < R; ++c)
          b[c][i] = v0 + 32 * i < nv ? __ldg(reinterpret_cast<const uint4*>(w[c]) + v0 + 32 * i) : zero;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint4 xv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          xv[m] = v0 + 32 * i < nv ? __ldg(reinterpret_cast<const uint4*>(x[m]) + v0 + 32 * i) : zero;
        float wf[R][E];
#pragma unroll
        for (int c = 0; c < R; ++c) unpack(b[c][i], wf[c], T());
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float xf[E];
          unpack(xv[m], xf, T());
#pragma unroll
          for (int c = 0; c < R; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[c][m] = fmaf(xf[e], wf[c][e], acc[c][m]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = min(v0 + 32 * i, a.K - 1);
        const bool in = v0 + 32 * i < nv;
        float wf[R];
#pragma unroll
        for (int c = 0; c < R; ++c) wf[c] = in ? elem(w[c][k]) : 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float xf = in ? elem(x[m][k]) : 0.f;
#pragma unroll
          for (int c = 0; c < R; ++c) acc[c][m] = fmaf(xf, wf[c], acc[c][m]);
        }
      }
    }
  }
  // lane m + MT c ends with row m's sums of column c
  constexpr int S = MT == 1 ? 1 : 8;
  float z[NB] = {};
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < R; ++c) {
      float v = acc[c][m];
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == m + S * (c % NC)) z[c / NC] = v;
    }
  const int n = n0 + lane / S;
  if (lane % S >= rows || lane >= S * NC || n >= a.N) return;
  const long long m = m0 + lane % S;
#pragma unroll
  for (int h = 0; h < NB; ++h) {
    if (a.xs) z[h] *= a.xs[m] * a.ws[n + h * a.N];
    if (a.bias) z[h] += a.bias[n + h * a.N];
  }
  float r = act_any(a.act, z[0]);
  if (GATED) r *= z[NB - 1];
  if (a.res) r += elem(static_cast<const TO*>(a.res)[m * a.ldr + n]);
  static_cast<TO*>(a.y)[m * a.ldy + n] = TO(r);
}

template <class T, class TO, int MT, int NC, bool GATED>
bool launch_small_v(SmallArgs a, bool vec, cudaStream_t s) {
  a.col_blocks = (a.N + 8 * NC - 1) / (8 * NC);
  const dim3 grid(unsigned(a.col_blocks) * unsigned((a.M + MT - 1) / MT));
  if (!vec) return pdl_launch(small_kernel<T, TO, MT, NC, GATED, false, false>, grid, 256, s, a);
  return a.K * int(sizeof(T)) <= 512 ? pdl_launch(small_kernel<T, TO, MT, NC, GATED, true, true>, grid, 256, s, a)
                                     : pdl_launch(small_kernel<T, TO, MT, NC, GATED, true, false>, grid, 256, s, a);
}
// Columns per warp: as many as leave the chip about five warps per SM. (8 x
// 1024 -> 4096: 6.5 us with four columns, 8.7 with one in bf16, 10.7 and 16.3
// in fp32; 16 x 1024 -> 1024: 6.9 us with two, 5.6 with one.)
inline int small_columns(const SmallArgs& a) {
  constexpr long long kMinWarps = 800;
  const long long chunks = (a.M + kSmallM - 1) / kSmallM;
  return a.N * chunks >= 4 * kMinWarps ? 4 : (a.N * chunks >= 2 * kMinWarps ? 2 : 1);
}

// Whether a forward call takes this kernel: up to 8 rows, or a product small
// enough that the tensor-core kernel's fixed cost (4 to 5 us; fp32 8 to 10 with
// the terms laid out) is more than all of it. Measured around the borders
// (multiplies; this kernel, the other): bf16 16.8 M 3.7 and 4.6 us, 33.6 M 6.5
// and 4.7; fp32 33.6 M 9.7 and 9.8, 67 M 11.5 to 16.9 and 10.2 to 13.1; e4m3
// 8.4 M 3.1 and 4.1, 16.8 M 5.5 and 4.3.
inline bool small_call(int dtype, long long M, int R, int K) {
  const double most = dtype == DSF_F32 ? 1 << 25 : (dtype == DSF_BF16 ? 1 << 24 : 1 << 23);
  return M <= kSmallM || double(M) * R * K <= most;
}
template <class T, class TO, bool GATED>
bool launch_small_g(const SmallArgs& a, bool vec, cudaStream_t s) {
  if (a.M == 1) return launch_small_v<T, TO, 1, 1, GATED>(a, vec, s);
  const int nc = small_columns(a);
  if (nc == 4 && !GATED) return launch_small_v<T, TO, kSmallM, 4, GATED>(a, vec, s);
  return nc >= 2 ? launch_small_v<T, TO, kSmallM, 2, GATED>(a, vec, s)
                 : launch_small_v<T, TO, kSmallM, 1, GATED>(a, vec, s);
}
template <class T, class TO>
bool launch_small(const SmallArgs& a, bool gated, bool vec, cudaStream_t s) {
  return gated ? launch_small_g<T, TO, true>(a, vec, s) : launch_small_g<T, TO, false>(a, vec, s);
}

}  // namespace dense
}  // namespace dsf
