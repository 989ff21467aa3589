// The root-mean-square norm of the dense towers: s = x + residual (rounded to
// x's type, as later layers read it), y = s w / sqrt(mean(s^2) + eps), with an
// optional 8-bit output (e4m3 values and one scale per row), and its gradient.
//
// Both directions are bound by HBM: a row is read once, held in registers
// between the row sum and the outputs, and written once. A row belongs to a
// group of G threads -- one warp up to N = 1024 (bf16) or 512 (fp32), so that
// the row sums are warp shuffles and several rows are in flight per block,
// then 64 .. 1024 threads -- and each thread holds 8 V elements of it (V <= 4).
// Aligned rows move in 16-byte vectors, eight elements a thread; others (odd N,
// odd strides) element by element, the group's threads side by side.
// Measured: 65536 x 1024 bf16 with the residual to e4m3 71 us, 6.6 TB/s of
// algorithmic bytes (a plain copy of this chip: 6.8); its backward in bf16 72 us
// with the weight's gradient, 68 without.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "colsum.cuh"
#include "dinsparse.h"
#include "pdl.cuh"

namespace dsf {
namespace norm {
namespace {

constexpr int kMaxN = 32768;
constexpr int kBlock = 256;          // threads per block (a wider group is its own block)
constexpr int kSms = 152;
constexpr float kE4m3Max = 448.f;

struct FwdArgs {
  const void *x, *res;
  long long ldx, ldr;
  const float* w;
  long long M;
  int N;
  float eps;
  void* sum;
  long long lds;
  void* y;
  long long ldy;
  float* scale;
};

struct BwdArgs {
  const void *dy, *s, *dsum;
  long long lddy, lds, ldds;
  const float* w;
  long long M;
  int N;
  float eps;
  void* dx;
  long long lddx;
  float* part;  // [blocks][N], nullable
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// eight consecutive elements, 16-byte aligned (e4m3: 8 bytes)
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(u[k] << 16);
    v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    u[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ uint2 pack8_e4m3(const float* v) {
  uint32_t u[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k], v[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2], v[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
    u[k] = lo | hi << 16;
  }
  return make_uint2(u[0], u[1]);
}

// A group's share of a row: V sets of 8 elements per thread. ALIGNED: set i of
// thread t is the 8 consecutive elements from 8 (t + i G); else its elements
// are t, t + G, ... so that the group reads neighbouring elements.
template <bool ALIGNED, int G, class T>
__device__ __forceinline__ void load_set(const T* row, int i, int t, int N, float* v) {
  if (ALIGNED) {
    const int e = 8 * (t + i * G);
    if (e < N) {
      load8(row + e, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = (8 * i + j) * G + t;
      v[j] = e < N ? to_f(row[e]) : 0.f;
    }
  }
}
template <bool ALIGNED, int G, class T>
__device__ __forceinline__ void store_set(T* row, int i, int t, int N, const float* v) {
  if (ALIGNED) {
    const int e = 8 * (t + i * G);
    if (e < N) store8(row + e, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = (8 * i + j) * G + t;
      if (e < N) row[e] = from_f<T>(v[j]);
    }
  }
}

// Sum (or maximum) over the group's threads, the same bits in each. G > 32:
// the group is the whole block; buf: G / 32 words of shared memory that no
// other reduction in flight uses.
template <int G, bool MAX>
__device__ __forceinline__ float group_reduce(float v, float* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if (G == 32) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
#pragma unroll
  for (int k = 1; k < G / 32; ++k) v = MAX ? fmaxf(v, buf[k]) : v + buf[k];
  return v;
}

// Two sums at once.
template <int G>
__device__ __forceinline__ void group_reduce2(float& a, float& b, float* buf_a, float* buf_b) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (G == 32) return;
  if ((threadIdx.x & 31) == 0) {
    buf_a[threadIdx.x >> 5] = a;
    buf_b[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  a = buf_a[0];
  b = buf_b[0];
#pragma unroll
  for (int k = 1; k < G / 32; ++k) {
    a += buf_a[k];
    b += buf_b[k];
  }
}

// v / scale in e4m3, eight values. lo and hi are the rounded 1 / scale times 1 -
// 2^-22 and 1 + 2^-22, so that a product with one of them is below the quotient
// and one with the other above (four roundings of 2^-24 lie between). Where
// both round to the same e4m3 value, so does the quotient; else, next to a
// border, all eight are divided. That is rare with a weight; without one, bf16
// rows often hold values in a ratio to their largest that is a border exactly.
// (65536 x 1024 bf16 with the residual: 71 us with a weight, 78 without; 75 by
// the product with the rounded 1 / scale alone, which is wrong once in 4 million
// values with a weight and 2600 times without; 80 by divisions.)
__device__ __forceinline__ uint2 quotients8(const float* v, float scale, float lo, float hi) {
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = v[j] * lo;
    b[j] = v[j] * hi;
  }
  const uint2 q = pack8_e4m3(a), u = pack8_e4m3(b);
  if (q.x == u.x && q.y == u.y) return q;
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = v[j] / scale;
  return pack8_e4m3(a);
}
// The set of eight e4m3 values, as store_set.
template <bool ALIGNED, int G>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int i, int t, int N, uint2 q) {
  if (ALIGNED) {
    const int e = 8 * (t + i * G);
    if (e < N) *reinterpret_cast<uint2*>(row + e) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = (8 * i + j) * G + t;
      if (e < N) row[e] = uint8_t((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
    }
  }
}

template <class TX, class TY, int G, int V, bool ALIGNED>
__global__ void __launch_bounds__(G > kBlock ? G : kBlock) fwd_kernel(const FwdArgs a) {
  constexpr int T = G == 32 ? kBlock : G, RPB = T / G;
  __shared__ float buf[2][32];
  pdl_go();
  pdl_wait();
  const int t = threadIdx.x % G;
  const long long row = (long long)blockIdx.x * RPB + threadIdx.x / G;
  if (row >= a.M) return;  // (a whole warp or the whole block)
  const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
  float s[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) load_set<ALIGNED, G>(x, i, t, a.N, s[i]);
  if (a.res) {
    const TX* r = static_cast<const TX*>(a.res) + row * a.ldr;
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) load_set<ALIGNED, G>(r, i, t, a.N, v[i]);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = to_f(from_f<TX>(s[i][j] + v[i][j]));
  }
  if (a.sum) {
    TX* o = static_cast<TX*>(a.sum) + row * a.lds;
#pragma unroll
    for (int i = 0; i < V; ++i) store_set<ALIGNED, G>(o, i, t, a.N, s[i]);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(s[i][j], s[i][j], ss);
  ss = group_reduce<G, false>(ss, buf[0]);
  const float r = 1.f / sqrtf(ss / float(a.N) + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float w[8];
    if (a.w) {
      load_set<ALIGNED, G>(a.w, i, t, a.N, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * r * w[j];
  }
  TY* y = static_cast<TY*>(a.y) + row * a.ldy;
  if constexpr (sizeof(TY) == 1) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(s[i][j]));
    m = group_reduce<G, true>(m, buf[1]);
    const float scale = fmaxf(m / kE4m3Max, 1.17549435e-38f), inv = 1.f / scale;
    if (t == 0) a.scale[row] = scale;
    const float lo = inv * (1.f - 0x1p-22f), hi = inv * (1.f + 0x1p-22f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      store_e4m3<ALIGNED, G>(reinterpret_cast<uint8_t*>(y), i, t, a.N, quotients8(s[i], scale, lo, hi));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) store_set<ALIGNED, G>(y, i, t, a.N, s[i]);
  }
}

// A set of 8 elements as it is stored: two per register in bf16.
template <class T>
struct Pack {
  uint32_t w[2 * sizeof(T)];
};
__device__ __forceinline__ void open(const Pack<float>& p, float* v) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(p.w[k]);
}
__device__ __forceinline__ void open(const Pack<__nv_bfloat16>& p, float* v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(p.w[k] << 16);
    v[2 * k + 1] = __uint_as_float(p.w[k] & 0xffff0000u);
  }
}
template <bool ALIGNED, int G, class T>
__device__ __forceinline__ void load_pack(const T* row, int i, int t, int N, Pack<T>& p) {
  constexpr int W = 2 * int(sizeof(T));
#pragma unroll
  for (int k = 0; k < W; ++k) p.w[k] = 0;
  if (ALIGNED) {
    const int e = 8 * (t + i * G);
    if (e < N) {
#pragma unroll
      for (int k = 0; k < W / 4; ++k) {
        const uint4 u = reinterpret_cast<const uint4*>(row + e)[k];
        p.w[4 * k] = u.x, p.w[4 * k + 1] = u.y, p.w[4 * k + 2] = u.z, p.w[4 * k + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = (8 * i + j) * G + t;
      const uint32_t u = e < N ? __float_as_uint(to_f(row[e])) : 0u;
      if (sizeof(T) == 4) p.w[j % W] = u;
      else p.w[j / 2] |= j & 1 ? u : u >> 16;
    }
  }
}
template <bool ALIGNED, int G>
__device__ __forceinline__ void load_weight(const float* w, int i, int t, int N, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = w ? 0.f : 1.f;
  if (!w) return;
  if (ALIGNED) {
    const int e = 8 * (t + i * G);
    if (e >= N) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(w + e) + k);
      v[4 * k] = x.x, v[4 * k + 1] = x.y, v[4 * k + 2] = x.z, v[4 * k + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = (8 * i + j) * G + t;
      if (e < N) v[j] = __ldg(w + e);
    }
  }
}

// dx = r (g - s r^2 mean(g s)) + dsum with g = dy w and r = 1 / sqrt(mean(s^2)
// + eps): both row sums come from one reading of s and dy, which wait in
// registers as they are stored (the weight is read twice, from L1). Blocks
// walk the rows, so that a thread's weight-gradient sums (dy s r of its
// columns) stay in registers over all of them; a block then writes one row of
// partial sums. Blocks of up to 256 threads have 128 registers a thread, so that
// 512 threads fit an SM: with the operands held as fp32 256 did, and 65536 x
// 1024 in bf16 took 99 us where HBM needs 59. (Wider groups, one row per block,
// have what 512 or 1024 threads leave, and spill: fp32 rows of 16384 take 57 us
// per 1000 where HBM needs 29, of 32768 82 us per 500.)
template <class TY, class TX, int G, int V, bool ALIGNED>
__global__ void __launch_bounds__(G > kBlock ? G : kBlock, G > kBlock ? 1 : 2) bwd_kernel(const BwdArgs a) {
  constexpr int T = G == 32 ? kBlock : G, RPB = T / G;
  __shared__ float buf[2][2][32];
  __shared__ float wsum[G == 32 ? RPB : 1][G == 32 ? 8 * V * 32 : 1];
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  pdl_go();
  pdl_wait();
  int par = 0;  // two sets of reduction buffers: a row's writes never meet the last row's reads
  for (long long row = (long long)blockIdx.x * RPB + grp; row < a.M; row += (long long)gridDim.x * RPB, par ^= 1) {
    Pack<TX> sp[V];
    Pack<TY> dp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) load_pack<ALIGNED, G>(static_cast<const TX*>(a.s) + row * a.lds, i, t, a.N, sp[i]);
#pragma unroll
    for (int i = 0; i < V; ++i) load_pack<ALIGNED, G>(static_cast<const TY*>(a.dy) + row * a.lddy, i, t, a.N, dp[i]);
    float ss = 0.f, gs = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s[8], d[8], w[8];
      open(sp[i], s);
      open(dp[i], d);
      load_weight<ALIGNED, G>(a.w, i, t, a.N, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(s[j], s[j], ss);
        gs = fmaf(d[j] * w[j], s[j], gs);
      }
    }
    group_reduce2<G>(ss, gs, buf[par][0], buf[par][1]);
    const float r = 1.f / sqrtf(ss / float(a.N) + a.eps);
    const float c = r * r * (gs / float(a.N));
    TX* o = static_cast<TX*>(a.dx) + row * a.lddx;
    const TX* u = static_cast<const TX*>(a.dsum) + row * a.ldds;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s[8], d[8], w[8];
      open(sp[i], s);
      open(dp[i], d);
      load_weight<ALIGNED, G>(a.w, i, t, a.N, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[i][j] = fmaf(d[j] * r, s[j], dw[i][j]);
        d[j] = r * (d[j] * w[j] - s[j] * c);
      }
      if (a.dsum) {
        float v[8];
        load_set<ALIGNED, G>(u, i, t, a.N, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += v[j];
      }
      store_set<ALIGNED, G>(o, i, t, a.N, d);
    }
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * a.N;
  if (G == 32) {  // the block's warps add up in shared memory, in warp order
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) wsum[grp][(ALIGNED ? 8 * (t + i * G) + j : (8 * i + j) * G + t)] = dw[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.N; e += T) {
      float v = wsum[0][e];
#pragma unroll
      for (int k = 1; k < RPB; ++k) v += wsum[k][e];
      out[e] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) store_set<ALIGNED, G>(out, i, t, a.N, dw[i]);
  }
}

// One variant per row length: (G, V) with 8 G V >= N, the smallest group first
// (a longer row takes more sets per thread, then more threads).
template <class F>
bool by_length(int N, F&& f) {
  if (N <= 256) return f.template operator()<32, 1>();
  if (N <= 512) return f.template operator()<32, 2>();
  if (N <= 1024) return f.template operator()<32, 4>();
  if (N <= 2048) return f.template operator()<128, 2>();
  if (N <= 4096) return f.template operator()<128, 4>();
  if (N <= 8192) return f.template operator()<256, 4>();
  if (N <= 16384) return f.template operator()<512, 4>();
  return f.template operator()<1024, 4>();
}

// Rows of fp32 (in the backward: either operand) take twice the registers per
// element: two sets per thread at most, as far as 1024 threads go. (8192 x 1024
// in fp32: forward 12.1 us; backward 18.0, 21.3 with the weight's gradient.)
template <class F>
bool by_length_wide(int N, F&& f) {
  if (N <= 256) return f.template operator()<32, 1>();
  if (N <= 512) return f.template operator()<32, 2>();
  if (N <= 1024) return f.template operator()<64, 2>();
  if (N <= 2048) return f.template operator()<128, 2>();
  if (N <= 4096) return f.template operator()<256, 2>();
  if (N <= 8192) return f.template operator()<512, 2>();
  if (N <= 16384) return f.template operator()<1024, 2>();
  return f.template operator()<1024, 4>();
}

bool aligned_rows(const void* p, long long ld, int es) {
  return !p || ((reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * es) % 16 == 0);
}

int esize(int dtype) { return dtype == DSF_F32 ? 4 : (dtype == DSF_BF16 ? 2 : 1); }

// Blocks of the backward for rows in groups of G, each with one row of
// weight-gradient sums: 8 rows at a time each where a row is a warp's, else one,
// as many as are resident at 512 threads per SM (two blocks of 256, four of
// 128, eight of 64).
template <int G>
long long bwd_blocks(long long M) {
  constexpr int T = G == 32 ? kBlock : G, RPB = T / G;
  const long long b = (M + RPB - 1) / RPB, most = kSms * (T < 512 ? 512 / T : 1);
  return b < most ? b : most;
}

// What by_length and by_length_wide are given to learn a variant's blocks.
struct BwdBlocks {
  long long M;
  long long* blocks;
  template <int G, int V>
  bool operator()() const {
    *blocks = bwd_blocks<G>(M);
    return true;
  }
};

// Rows of partial sums of a backward call, whatever its operands' types are.
long long part_rows(long long M, int N) {
  long long a = 0, b = 0;
  by_length(N, BwdBlocks{M, &a});
  by_length_wide(N, BwdBlocks{M, &b});
  return a > b ? a : b;
}

template <class TX, class TY>
struct Fwd {
  const FwdArgs& a;
  bool al;
  cudaStream_t st;
  template <int G, int V>
  bool operator()() const {
    constexpr int T = G == 32 ? kBlock : G, RPB = T / G;
    const unsigned grid = unsigned((a.M + RPB - 1) / RPB);
    return pdl_launch(al ? fwd_kernel<TX, TY, G, V, true> : fwd_kernel<TX, TY, G, V, false>, dim3(grid), T, st, a);
  }
};
template <class TY, class TX>
struct Bwd {
  const BwdArgs& a;
  bool al;
  cudaStream_t st;
  long long* blocks;  // out: the rows of partial sums
  template <int G, int V>
  bool operator()() const {
    constexpr int T = G == 32 ? kBlock : G;
    *blocks = bwd_blocks<G>(a.M);
    return pdl_launch(al ? bwd_kernel<TY, TX, G, V, true> : bwd_kernel<TY, TX, G, V, false>, dim3(unsigned(*blocks)), T,
                      st, a);
  }
};

bool elem_aligned(const void* p, int es) { return (reinterpret_cast<uintptr_t>(p) % es) == 0; }

}  // namespace
}  // namespace norm
}  // namespace dsf

using namespace dsf;
using namespace dsf::norm;

extern "C" {

int ctr_rms_norm_fwd(const void* x, int64_t ldx, const void* res, int64_t ldr, int32_t x_dtype, const float* w,
                     int64_t M, int32_t N, float eps, void* sum, int64_t lds, void* y, int64_t ldy, int32_t y_dtype,
                     float* y_scale, void* stream) {
  if (M < 0 || M > INT32_MAX || N < 1 || !(eps > 0.f)) return DSF_EINVAL;
  if (N > kMaxN) return DSF_EUNSUPPORTED;
  if (x_dtype != DSF_F32 && x_dtype != DSF_BF16) return DSF_EUNSUPPORTED;
  if (y_dtype != DSF_F32 && y_dtype != DSF_BF16 && y_dtype != DSF_E4M3) return DSF_EUNSUPPORTED;
  if (M == 0) return DSF_OK;
  const int ex = esize(x_dtype), ey = esize(y_dtype);
  if (!x || !y || ldx < N || ldy < N || (res && ldr < N) || (sum && lds < N)) return DSF_EINVAL;
  if (!elem_aligned(x, ex) || !elem_aligned(res, ex) || !elem_aligned(sum, ex) || !elem_aligned(y, ey) ||
      !elem_aligned(w, 4) || !elem_aligned(y_scale, 4))
    return DSF_EINVAL;
  if ((y_dtype == DSF_E4M3) != (y_scale != nullptr)) return DSF_EINVAL;
  const FwdArgs a{x, res, ldx, ldr, w, M, N, eps, sum, lds, y, ldy, y_scale};
  const bool al = N % 8 == 0 && aligned_rows(x, ldx, ex) && aligned_rows(res, ldr, ex) &&
                  aligned_rows(sum, lds, ex) && aligned_rows(w, 0, 4) &&
                  (y_dtype == DSF_E4M3 ? (reinterpret_cast<uintptr_t>(y) % 8 == 0 && ldy % 8 == 0)
                                       : aligned_rows(y, ldy, ey));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bool ok;
  if (x_dtype == DSF_F32) {
    if (y_dtype == DSF_F32) ok = by_length_wide(N, Fwd<float, float>{a, al, st});
    else if (y_dtype == DSF_BF16) ok = by_length_wide(N, Fwd<float, __nv_bfloat16>{a, al, st});
    else ok = by_length_wide(N, Fwd<float, __nv_fp8_e4m3>{a, al, st});
  } else {
    if (y_dtype == DSF_F32) ok = by_length(N, Fwd<__nv_bfloat16, float>{a, al, st});
    else if (y_dtype == DSF_BF16) ok = by_length(N, Fwd<__nv_bfloat16, __nv_bfloat16>{a, al, st});
    else ok = by_length(N, Fwd<__nv_bfloat16, __nv_fp8_e4m3>{a, al, st});
  }
  return ok ? DSF_OK : DSF_ECUDA;
}

size_t dsf_rms_norm_workspace_bytes(int64_t M, int32_t N) {
  if (M < 0 || M > INT32_MAX || N < 1 || N > kMaxN) return 0;
  const long long b = part_rows(M, N);
  return (size_t(b > 0 ? b : 1) * N * 4 + 255) / 256 * 256;
}

int ctr_rms_norm_bwd(const void* dy, int64_t lddy, int32_t dy_dtype, const void* s, int64_t lds, int32_t x_dtype,
                     const float* w, int64_t M, int32_t N, float eps, const void* dsum, int64_t ldds, void* dx,
                     int64_t lddx, float* dw, void* ws, size_t ws_bytes, void* stream) {
  if (M < 0 || M > INT32_MAX || N < 1 || !(eps > 0.f)) return DSF_EINVAL;
  if (N > kMaxN) return DSF_EUNSUPPORTED;
  if (x_dtype != DSF_F32 && x_dtype != DSF_BF16) return DSF_EUNSUPPORTED;
  if (dy_dtype != DSF_F32 && dy_dtype != DSF_BF16) return DSF_EUNSUPPORTED;
  const int ex = esize(x_dtype), ey = esize(dy_dtype);
  if (!elem_aligned(dw, 4)) return DSF_EINVAL;
  if (dw && (!ws || (reinterpret_cast<uintptr_t>(ws) % 256) || ws_bytes < dsf_rms_norm_workspace_bytes(M, N)))
    return DSF_EWORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dw && !succeeded(cudaMemsetAsync(dw, 0, size_t(N) * 4, st))) return DSF_ECUDA;
    return DSF_OK;
  }
  if (!dy || !s || !dx || lddy < N || lds < N || lddx < N || (dsum && ldds < N)) return DSF_EINVAL;
  if (!elem_aligned(dy, ey) || !elem_aligned(s, ex) || !elem_aligned(dsum, ex) || !elem_aligned(dx, ex) ||
      !elem_aligned(w, 4))
    return DSF_EINVAL;
  const BwdArgs a{dy, s, dsum, lddy, lds, ldds, w, M, N, eps, dx, lddx, dw ? static_cast<float*>(ws) : nullptr};
  const bool al = N % 8 == 0 && aligned_rows(dy, lddy, ey) && aligned_rows(s, lds, ex) &&
                  aligned_rows(dsum, ldds, ex) && aligned_rows(dx, lddx, ex) && aligned_rows(w, 0, 4);
  bool ok;
  long long blocks = 0;
  if (dy_dtype == DSF_F32)
    ok = x_dtype == DSF_F32 ? by_length_wide(N, Bwd<float, float>{a, al, st, &blocks})
                            : by_length_wide(N, Bwd<float, __nv_bfloat16>{a, al, st, &blocks});
  else
    ok = x_dtype == DSF_F32 ? by_length_wide(N, Bwd<__nv_bfloat16, float>{a, al, st, &blocks})
                            : by_length(N, Bwd<__nv_bfloat16, __nv_bfloat16>{a, al, st, &blocks});
  if (!ok) return DSF_ECUDA;
  if (dw && !colsum(a.part, blocks, N, dw, st)) return DSF_ECUDA;
  return DSF_OK;
}

}  // extern "C"
