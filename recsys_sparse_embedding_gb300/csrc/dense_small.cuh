// Forward of a few rows (M <= 8): the weights are read once, straight from
// memory, on the CUDA cores.
//
// y[m][n] = sum over k of x[m][k] W[n][k] needs 2 M operations per weight, so
// up to a handful of rows the weights' bytes are all that counts: a tensor-core
// tile would use 8 of its 128 rows. A warp takes one output column (a gated
// layer: its gate and up rows), its lanes side by side along K in 16-byte
// vectors, four vectors in flight; x (a few KB) stays in L1. fp32 sums, then
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

template <class T, class TO, int MT, bool GATED, bool VEC>
__global__ void __launch_bounds__(256) small_kernel(const SmallArgs a) {
  constexpr int NB = GATED ? 2 : 1, E = VEC ? 16 / int(sizeof(T)) : 1, U = VEC ? 4 : 8;
  const int lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_go();
  pdl_wait();
  if (n >= a.N) return;
  const T* x = static_cast<const T*>(a.x);
  const T* w[NB];
#pragma unroll
  for (int h = 0; h < NB; ++h) w[h] = static_cast<const T*>(a.W) + (long long)(n + h * a.N) * a.ldw;
  float acc[NB][MT];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[h][m] = 0.f;
  const int nv = a.K / E;  // (VEC: K is a whole number of vectors)
  for (int v0 = lane; v0 < nv; v0 += 32 * U) {
    if constexpr (VEC) {
      uint4 b[NB][U];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < NB; ++h)
          b[h][i] = v0 + 32 * i < nv ? __ldg(reinterpret_cast<const uint4*>(w[h]) + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (v0 + 32 * i >= nv) break;
        float wf[NB][E];
#pragma unroll
        for (int h = 0; h < NB; ++h) unpack(b[h][i], wf[h], T());
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m >= a.M) break;
          float xf[E];
          unpack(__ldg(reinterpret_cast<const uint4*>(x + m * a.ldx) + v0 + 32 * i), xf, T());
#pragma unroll
          for (int h = 0; h < NB; ++h)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[h][m] = fmaf(xf[e], wf[h][e], acc[h][m]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = v0 + 32 * i;
        if (k >= nv) break;
        float wf[NB];
#pragma unroll
        for (int h = 0; h < NB; ++h) wf[h] = elem(w[h][k]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m >= a.M) break;
          const float xf = elem(x[m * a.ldx + k]);
#pragma unroll
          for (int h = 0; h < NB; ++h) acc[h][m] = fmaf(xf, wf[h], acc[h][m]);
        }
      }
    }
  }
  float z[NB] = {};  // row `lane`'s sums
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < NB; ++h) {
      float v = acc[h][m];
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == m) z[h] = v;
    }
  if (lane >= a.M) return;
#pragma unroll
  for (int h = 0; h < NB; ++h) {
    if (a.xs) z[h] *= a.xs[lane] * a.ws[n + h * a.N];
    if (a.bias) z[h] += a.bias[n + h * a.N];
  }
  float r = act_any(a.act, z[0]);
  if (GATED) r *= z[NB - 1];
  if (a.res) r += elem(static_cast<const TO*>(a.res)[lane * a.ldr + n]);
  static_cast<TO*>(a.y)[lane * a.ldy + n] = TO(r);
}

template <class T, class TO, int MT, bool GATED>
bool launch_small_v(const SmallArgs& a, bool vec, cudaStream_t s) {
  const dim3 grid(unsigned((a.N + 7) / 8));
  return vec ? pdl_launch(small_kernel<T, TO, MT, GATED, true>, grid, 256, s, a)
             : pdl_launch(small_kernel<T, TO, MT, GATED, false>, grid, 256, s, a);
}
template <class T, class TO>
bool launch_small(const SmallArgs& a, bool gated, bool vec, cudaStream_t s) {
  if (a.M == 1) return gated ? launch_small_v<T, TO, 1, true>(a, vec, s) : launch_small_v<T, TO, 1, false>(a, vec, s);
  return gated ? launch_small_v<T, TO, kSmallM, true>(a, vec, s) : launch_small_v<T, TO, kSmallM, false>(a, vec, s);
}

}  // namespace dense
}  // namespace dsf
