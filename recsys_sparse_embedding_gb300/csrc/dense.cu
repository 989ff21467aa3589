// The dense operators of any width (declared in dinsparse.h): argument checks,
// workspace layout and the kernels' launches.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "colsum.cuh"
#include "dense_math.cuh"
#include "dinsparse.h"

namespace dsf {
namespace dense {
namespace {

constexpr int kMaxDim = 1 << 20;
constexpr long long kMaxM = INT32_MAX - 1024;

int esize(int dtype) { return dtype == DSF_F32 ? 4 : (dtype == DSF_BF16 ? 2 : 1); }
int osize(int dtype) { return dtype == DSF_F32 ? 4 : 2; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool at(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of `cols` elements of es bytes: 16-byte boundaries are asked for where
// the row's own length keeps them.
bool rows_ok(const void* p, long long ld, long long cols, int es) {
  if (!p || ld < cols || !at(p, es)) return false;
  return (cols * es) % 16 != 0 || (at(p, 16) && (ld * es) % 16 == 0);
}

int check_layer(const dsf_dense* l, bool gated) {
  if (!l || !l->W) return DSF_EINVAL;
  if (l->dtype != DSF_F32 && l->dtype != DSF_BF16 && l->dtype != DSF_E4M3) return DSF_EUNSUPPORTED;
  if (l->act < DSF_ACT_NONE || l->act > DSF_ACT_GELU) return DSF_EINVAL;
  if (l->R < 1 || l->K < 1 || l->R > kMaxDim || l->K > kMaxDim || (gated && l->R % 2)) return DSF_EINVAL;
  if (!rows_ok(l->W, l->ldw, l->K, esize(l->dtype)) || !at(l->bias, 4)) return DSF_EINVAL;
  if ((l->dtype == DSF_E4M3) != (l->scale != nullptr) || !at(l->scale, 4)) return DSF_EINVAL;
  return DSF_OK;
}

// Workspace: dz of the backward in fp32, [M, R].
size_t ws_bytes_of(const dsf_dense* l, long long M, bool gated, bool backward) {
  return align256(256 + (backward ? size_t(M) * l->R * 4 : 0));
}

__device__ __forceinline__ float ld_f(const float* p) { return *p; }
__device__ __forceinline__ float ld_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld_f(const __nv_fp8_e4m3* p) { return float(*p); }
__device__ __forceinline__ void st_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// acc[m][n] = sum over k of A(m, k) B(n, k), tiles of 64 x 64 by 256 threads,
// K-steps of 16 through shared memory; epi(m, n, acc, acc of row n + gap).
template <class TA, class TB, bool GATED, class Epi>
__global__ void __launch_bounds__(256) product_kernel(const TA* A, long long am, long long ak, const TB* B,
                                                      long long bn, long long bk, long long M, int N, long long K,
                                                      int gap, const Epi epi) {
  constexpr int T = 64, BK = 16, NB = GATED ? 2 : 1;
  __shared__ float As[BK][T + 1], Bs[NB][BK][T + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const long long m0 = (long long)blockIdx.x * T;
  const int n0 = blockIdx.y * T;
  float acc[NB][4][4] = {};
  for (long long k0 = 0; k0 < K; k0 += BK) {
    for (int e = tid; e < T * BK; e += 256) {
      const int r = e / BK, c = e % BK;
      const long long k = k0 + c, m = m0 + r;
      const int n = n0 + r;
      As[c][r] = m < M && k < K ? ld_f(A + m * am + k * ak) : 0.f;
#pragma unroll
      for (int h = 0; h < NB; ++h)
        Bs[h][c][r] = n < N && k < K ? ld_f(B + (long long)(n + h * gap) * bn + k * bk) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < BK; ++c)
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[h][i][j] = fmaf(As[c][ty * 4 + i], Bs[h][c][tx * 4 + j], acc[h][i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty * 4 + i;
      const int n = n0 + tx * 4 + j;
      if (m < M && n < N) epi(m, n, acc[0][i][j], GATED ? acc[NB - 1][i][j] : 0.f);
    }
}

__device__ __forceinline__ float act_any(int act, float z) {
  return act == DSF_ACT_RELU ? act_value<DSF_ACT_RELU>(z)
                             : (act == DSF_ACT_SILU ? act_value<DSF_ACT_SILU>(z)
                                                    : (act == DSF_ACT_GELU ? act_value<DSF_ACT_GELU>(z) : z));
}
__device__ __forceinline__ float2 both_any(int act, float z) {
  return act == DSF_ACT_RELU
             ? act_both<DSF_ACT_RELU>(z)
             : (act == DSF_ACT_SILU ? act_both<DSF_ACT_SILU>(z)
                                    : (act == DSF_ACT_GELU ? act_both<DSF_ACT_GELU>(z) : make_float2(z, 1.f)));
}

template <class TO>
struct FwdEpi {
  TO* y;
  const TO* res;
  const float *bias, *xs, *ws;
  long long ldy, ldr;
  int act, gap;  // gap > 0: the gated layer, F
  __device__ float z(long long m, int n, float acc) const {
    if (xs) acc *= xs[m] * ws[n];
    return bias ? acc + bias[n] : acc;
  }
  __device__ void operator()(long long m, int n, float a, float b) const {
    float v = act_any(act, z(m, n, a));
    if (gap) v *= z(m, n + gap, b);
    if (res) v += ld_f(res + m * ldr + n);
    st_f(y + m * ldy + n, v);
  }
};

template <class T>
struct DzEpi {
  const T* dy;
  const float* bias;
  long long lddy;
  float* dz;  // [M][R]
  int act, gap, R;
  __device__ void operator()(long long m, int n, float a, float b) const {
    const float g = ld_f(dy + m * lddy + n);
    const float2 f = both_any(act, bias ? a + bias[n] : a);
    if (gap) {
      const float u = bias ? b + bias[n + gap] : b;
      dz[m * R + n] = g * u * f.y;
      dz[m * R + n + gap] = g * f.x;
    } else {
      dz[m * R + n] = g * f.y;
    }
  }
};

template <class T>
struct OutEpi {
  T* o;
  long long ld;
  __device__ void operator()(long long m, int n, float a, float) const { st_f(o + m * ld + n, a); }
};

template <class TA, class TB, bool GATED, class Epi>
bool product(const TA* A, long long am, long long ak, const TB* B, long long bn, long long bk, long long M, int N,
             long long K, int gap, const Epi& epi, cudaStream_t s) {
  product_kernel<TA, TB, GATED><<<dim3(unsigned((M + 63) / 64), unsigned((N + 63) / 64)), 256, 0, s>>>(
      A, am, ak, B, bn, bk, M, N, K, gap, epi);
  return cudaGetLastError() == cudaSuccess;
}

template <class T, class TO>
int fwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const float* xs, const void* res, long long ldr,
        long long M, void* y, long long ldy, cudaStream_t s) {
  const int N = gated ? l->R / 2 : l->R;
  const FwdEpi<TO> e{static_cast<TO*>(y), static_cast<const TO*>(res), l->bias, xs, l->scale, ldy, ldr, l->act,
                     gated ? N : 0};
  const T *X = static_cast<const T*>(x), *W = static_cast<const T*>(l->W);
  const bool ok = gated ? product<T, T, true>(X, ldx, 1, W, l->ldw, 1, M, N, l->K, N, e, s)
                        : product<T, T, false>(X, ldx, 1, W, l->ldw, 1, M, N, l->K, 0, e, s);
  return ok ? DSF_OK : DSF_ECUDA;
}

template <class T>
int bwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const void* dy, long long lddy, long long M,
        void* dx, long long lddx, void* dW, float* db, void* ws, cudaStream_t s) {
  const int R = l->R, N = gated ? R / 2 : R, K = l->K;
  float* dz = static_cast<float*>(ws);
  const T *X = static_cast<const T*>(x), *W = static_cast<const T*>(l->W);
  const DzEpi<T> e{static_cast<const T*>(dy), l->bias, lddy, dz, l->act, gated ? N : 0, R};
  bool ok = gated ? product<T, T, true>(X, ldx, 1, W, l->ldw, 1, M, N, K, N, e, s)
                  : product<T, T, false>(X, ldx, 1, W, l->ldw, 1, M, N, K, 0, e, s);
  if (ok && dx)
    ok = product<float, T, false>(dz, R, 1, W, 1, l->ldw, M, K, R, 0, OutEpi<T>{static_cast<T*>(dx), lddx}, s);
  if (ok && dW)
    ok = product<float, T, false>(dz, 1, R, X, 1, ldx, R, K, M, 0, OutEpi<T>{static_cast<T*>(dW), K}, s);
  if (ok && db) ok = colsum(dz, M, R, db, s);
  return ok ? DSF_OK : DSF_ECUDA;
}

int run_fwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const float* xs, const void* res,
            long long ldr, long long M, void* y, long long ldy, void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_layer(l, gated)) return rc;
  if (M < 0 || M > kMaxM) return DSF_EINVAL;
  if (M == 0) return DSF_OK;
  const int N = gated ? l->R / 2 : l->R, eo = osize(l->dtype);
  if (!rows_ok(x, ldx, l->K, esize(l->dtype))) return DSF_EINVAL;
  if ((l->dtype == DSF_E4M3) != (xs != nullptr) || !at(xs, 4)) return DSF_EINVAL;
  if (!y || ldy < N || !at(y, eo) || (res && (ldr < N || !at(res, eo)))) return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < ws_bytes_of(l, M, gated, false)) return DSF_EWORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (l->dtype == DSF_F32) return fwd<float, float>(l, gated, x, ldx, xs, res, ldr, M, y, ldy, s);
  if (l->dtype == DSF_BF16) return fwd<__nv_bfloat16, __nv_bfloat16>(l, gated, x, ldx, xs, res, ldr, M, y, ldy, s);
  return fwd<__nv_fp8_e4m3, __nv_bfloat16>(l, gated, x, ldx, xs, res, ldr, M, y, ldy, s);
}

int run_bwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const void* dy, long long lddy, long long M,
            void* dx, long long lddx, void* dW, float* db, void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_layer(l, gated)) return rc;
  if (l->dtype == DSF_E4M3) return DSF_EUNSUPPORTED;
  if (M < 0 || M > kMaxM) return DSF_EINVAL;
  const int N = gated ? l->R / 2 : l->R, es = esize(l->dtype);
  if (!at(dW, es) || !at(db, 4)) return DSF_EINVAL;
  if (M > 0 && (!rows_ok(x, ldx, l->K, es) || !rows_ok(dy, lddy, N, es) || (dx && (lddx < l->K || !at(dx, es)))))
    return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < ws_bytes_of(l, M, gated, true)) return DSF_EWORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dW && cudaMemsetAsync(dW, 0, size_t(l->R) * l->K * es, s) != cudaSuccess) return DSF_ECUDA;
    if (db && cudaMemsetAsync(db, 0, size_t(l->R) * 4, s) != cudaSuccess) return DSF_ECUDA;
    return DSF_OK;
  }
  if (l->dtype == DSF_F32) return bwd<float>(l, gated, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, s);
  return bwd<__nv_bfloat16>(l, gated, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, s);
}

}  // namespace
}  // namespace dense
}  // namespace dsf

using namespace dsf::dense;

extern "C" {

size_t dsf_dense_workspace_bytes(const dsf_dense* l, int64_t M, int32_t gated, int32_t backward) {
  if (check_layer(l, gated != 0) != DSF_OK || M < 0 || M > kMaxM || gated < 0 || gated > 1 || backward < 0 ||
      backward > 1)
    return 0;
  if (backward && l->dtype == DSF_E4M3) return 0;
  return ws_bytes_of(l, M, gated != 0, backward != 0);
}

int ctr_dense_fwd(const dsf_dense* l, const void* x, int64_t ldx, const float* xs, const void* res, int64_t ldr,
                  int64_t M, void* y, int64_t ldy, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_fwd(l, false, x, ldx, xs, res, ldr, M, y, ldy, ws, ws_bytes, stream);
}

int ctr_glu_fwd(const dsf_dense* l, const void* x, int64_t ldx, const float* xs, int64_t M, void* h, int64_t ldh,
                void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_fwd(l, true, x, ldx, xs, nullptr, 0, M, h, ldh, ws, ws_bytes, stream);
}

int ctr_dense_bwd(const dsf_dense* l, const void* x, int64_t ldx, const void* dy, int64_t lddy, int64_t M, void* dx,
                  int64_t lddx, void* dW, float* db, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_bwd(l, false, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, ws_bytes, stream);
}

int ctr_glu_bwd(const dsf_dense* l, const void* x, int64_t ldx, const void* dh, int64_t lddh, int64_t M, void* dx,
                int64_t lddx, void* dW, float* db, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_bwd(l, true, x, ldx, dh, lddh, M, dx, lddx, dW, db, ws, ws_bytes, stream);
}

}  // extern "C"
