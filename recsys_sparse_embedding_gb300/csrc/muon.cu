// The orthogonalised update of a dense matrix (ctr_muon_update in dinsparse.h):
//   m = mu m + g,  u = g + mu m (or m),  X = u / (|u| + 1e-7),
//   five times  A = X X^T,  X = (a I + b A + c A^2) X,
//   W = W - lr (weight_decay W + sqrt(max(1, R / C)) X).
// The odd polynomial a x + b x^3 + c x^5 acts on X's singular values and sends
// all of (0, 1] near 1, so X ends near the closest orthogonal matrix. (A = X^T X
// on the right where C < R: the products are on the shorter side, n.)
//
// A small singular value grows by a = 3.44 a step, 485 times in five, and with it
// what the products round. Where W is fp32, X, A and the polynomial are fp32 taken as
// three bf16 terms each (six products of terms; X ends 1e-6 to 1e-5 off, as in fp32
// throughout). A bf16 W is rounded to 2^-9 in the end: two terms (2^-17, three
// products) leave X 2.5e-5 to 5e-5 off, which W's rounding hides at half the work.
// (One bf16 product would leave 1 to 3% of X, one fp16 0.2 to 0.3%.)
//
// A step's three products (2 n^2 m, 2 n^3 and 2 n^2 m operations) each leave fp32
// partial sums that a second kernel adds up and lays out as the next operand's terms.
#include "dense_host.cuh"

namespace dsf {
namespace dense {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f, kEps = 1e-7f;
constexpr int kMaxShort = 1 << 15, kMaxSteps = 16;
constexpr int kNormBlocks = 512;

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

// Four neighbouring elements of a matrix [R][ld], from column 4 j (fewer at a
// row's end).
template <class T>
__device__ __forceinline__ void get4(const T* p, int n, bool vec, float* v) {
  if (vec && n == 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
      v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = k < n ? elem(p[k]) : 0.f;
}
template <class T>
__device__ __forceinline__ void put4(T* p, int n, bool vec, const float* v) {
  if (vec && n == 4) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) put(p + k, v[k]);
}
// the three bf16 terms of four values, or the two nearest
__device__ __forceinline__ void put_terms(__nv_bfloat16* p, long long plane, const float* v, bool two) {
  float x[4] = {v[0], v[1], v[2], v[3]};
  if (two) {
    uint2 h = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    *reinterpret_cast<uint2*>(p) = h;
    const float l[4] = {x[0] - __uint_as_float(h.x << 16), x[1] - __uint_as_float(h.x & 0xffff0000u),
                        x[2] - __uint_as_float(h.y << 16), x[3] - __uint_as_float(h.y & 0xffff0000u)};
    *reinterpret_cast<uint2*>(p + plane) = make_uint2(pack_bf16x2(l[0], l[1]), pack_bf16x2(l[2], l[3]));
    return;
  }
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint32_t h[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = take_term(x[2 * k]), hi = take_term(x[2 * k + 1]);
      h[k] = __byte_perm(lo, hi, 0x7632);
    }
    *reinterpret_cast<uint2*>(p + t * plane) = make_uint2(h[0], h[1]);
  }
}

__device__ __forceinline__ float block_sum(float v, float* part) {  // 256 threads, in a fixed tree
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += part[w];
  __syncthreads();
  return s;
}

struct MomentArgs {
  const void* g;
  float *m, *u;     // u: [R][ldu]
  float* squares;   // a block's sum of u^2
  long long ldg, ldu;
  int R, C, n4;
  bool g_vec, m_vec, nesterov;
  float mu;
};
template <class TG>
__global__ void __launch_bounds__(256) moment_kernel(const __grid_constant__ MomentArgs a) {
  __shared__ float part[8];
  pdl_go();
  pdl_wait();
  float s = 0.f;
  const long long total = (long long)a.R * a.n4;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long r = i / a.n4;
    const int c = int(i - r * a.n4) * 4, n = min(4, a.C - c);
    float g[4], m[4], u[4];
    get4(static_cast<const TG*>(a.g) + r * a.ldg + c, n, a.g_vec, g);
    get4(a.m + r * a.C + c, n, a.m_vec, m);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = fmaf(a.mu, m[k], g[k]);
      u[k] = k < n ? (a.nesterov ? fmaf(a.mu, m[k], g[k]) : m[k]) : 0.f;
      s = fmaf(u[k], u[k], s);
    }
    put4(a.m + r * a.C + c, n, a.m_vec, m);
    put4(a.u + r * a.ldu + c, 4, true, u);
  }
  s = block_sum(s, part);
  if (threadIdx.x == 0) a.squares[blockIdx.x] = s;
}

// X = u / (|u| + eps), as terms
struct ScaleArgs {
  const float *u, *squares;
  __nv_bfloat16* x;
  long long ldu, ldx, plane;
  int R, n4, blocks;
  bool two;
};
__global__ void __launch_bounds__(256) scale_kernel(const __grid_constant__ ScaleArgs a) {
  __shared__ float part[8];
  pdl_go();
  pdl_wait();
  float s = 0.f;
  for (int i = threadIdx.x; i < a.blocks; i += 256) s += a.squares[i];
  const float d = sqrtf(block_sum(s, part)) + kEps;
  const long long total = (long long)a.R * a.n4;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long r = i / a.n4;
    const int c = int(i - r * a.n4) * 4;
    const float4 u = *reinterpret_cast<const float4*>(a.u + r * a.ldu + c);
    const float v[4] = {u.x / d, u.y / d, u.z / d, u.w / d};
    put_terms(a.x + r * a.ldx + c, a.plane, v, a.two);
  }
}

// A product's partial sums [splits][M][ldp] added in order, then
//   kSum   as terms, and in fp32 where f32 is given;
//   kPoly  a I + b A + c (the sum), A = f32, as terms;
//   kStep  W = decay W - rate (the sum).
enum { kSum = 0, kPoly = 1, kStep = 2 };
struct JoinArgs {
  const float* part;
  long long ldp, plane;
  int splits, M, N, n4;
  float* f32;  // [M][ldp]
  __nv_bfloat16* terms;
  long long ldt, tplane;
  void* W;
  long long ldw;
  bool w_vec, two;
  float decay, rate;
};
template <int MODE, class TW>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
  pdl_go();
  pdl_wait();
  const long long total = (long long)a.M * a.n4;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long r = i / a.n4;
    const int c = int(i - r * a.n4) * 4, n = min(4, a.N - c);
    float v[4] = {};
    const float* p = a.part + r * a.ldp + c;
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {
      const float4 f = *reinterpret_cast<const float4*>(p + z * a.plane);
      v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
    }
    if (MODE == kStep) {
      float w[4];
      TW* q = static_cast<TW*>(a.W) + r * a.ldw + c;
      get4(q, n, a.w_vec, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = fmaf(-a.rate, v[k], a.decay * w[k]);
      put4(q, n, a.w_vec, w);
      continue;
    }
    if (MODE == kPoly) {
      const float4 f = *reinterpret_cast<const float4*>(a.f32 + r * a.ldp + c);
      const float A[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fmaf(kC, v[k], kB * A[k]) + (r == c + k ? kA : 0.f);
    } else if (a.f32) {
      *reinterpret_cast<float4*>(a.f32 + r * a.ldp + c) = make_float4(v[0], v[1], v[2], v[3]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k >= n) v[k] = 0.f;
    put_terms(a.terms + r * a.ldt + c, a.tplane, v, a.two);
  }
}

struct MuonLayout {
  size_t x, a_terms, b_terms, a, u, squares, part, total;
  long long ldx, lda, R, C, n;
};
MuonLayout muon_layout(long long R, long long C) {
  MuonLayout w{};
  w.R = R, w.C = C, w.n = R < C ? R : C;
  w.ldx = up(C, 8), w.lda = up(w.n, 8);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t here = o;
    o += align256(bytes);
    return here;
  };
  auto part_of = [](size_t outputs) {
    const size_t all = outputs * 4 * kMaxSplits, may = all < kPartBytes ? all : kPartBytes;
    return may > outputs * 4 ? may : outputs * 4;
  };
  const size_t px = part_of(size_t(R) * w.ldx), pa = part_of(size_t(w.n) * w.lda);
  w.x = take(size_t(R) * w.ldx * 6);
  w.a_terms = take(size_t(w.n) * w.lda * 6);
  w.b_terms = take(size_t(w.n) * w.lda * 6);
  w.a = take(size_t(w.n) * w.lda * 4);
  w.squares = take(kNormBlocks * 4);
  w.part = take(px > pa ? px : pa);  // (u takes its place before the first product)
  w.u = w.part;
  w.total = o + 256;
  return w;
}

unsigned blocks_for(long long items) {
  const long long b = (items + 255) / 256;
  return unsigned(b < 1 ? 1 : (b < kSms * 8 ? b : kSms * 8));
}

// The product's partial sums to w.part.
bool part_product(Product& p, bool two, int major, const Mat& A, const Mat& B, long long M, long long N, long long K,
                  uint8_t* ws, const MuonLayout& w, int* status, cudaStream_t s) {
  p = Product{};
  p.major = major;
  p.f32 = !two;
  p.two = two;
  p.epi = kEpiOut;
  plan(p, M, N, 1, (K + 63) / 64, 1, true);
  p.epi = kEpiPart;
  p.A = A;
  p.B = B;
  p.a.status = status;
  Job& o = p.a.job[0];
  o.a_term = o.b_term = 1;
  o.out = ws + w.part;
  o.ldo = up(N, 4);
  o.out_plane = M * o.ldo;
  o.out_vec = 1;
  return two ? run_two_product(p, s) : (major == kKK ? run_fwd_product(p, s) : run_grad_product(p, s));
}

template <int MODE, class TW>
bool join(const Product& p, JoinArgs j, uint8_t* ws, const MuonLayout& w, cudaStream_t s) {
  const Job& o = p.a.job[0];
  j.part = reinterpret_cast<const float*>(ws + w.part);
  j.ldp = o.ldo;
  j.plane = o.out_plane;
  j.splits = o.splits;
  j.M = o.M;
  j.N = o.N;
  j.n4 = int(o.ldo / 4);
  j.two = p.two;
  return pdl_launch(join_kernel<MODE, TW>, dim3(blocks_for((long long)j.M * j.n4)), 256, s, j);
}

struct Step {
  void* W;
  long long ldw;
  int w_dtype;
  const void* g;
  long long ldg;
  int g_dtype;
  float* m;
  float lr, mu, decay;
  bool nesterov;
  int steps;
};

bool muon(const Step& q, long long R, long long C, uint8_t* ws, int* status, cudaStream_t s) {
  const MuonLayout w = muon_layout(R, C);
  const int n4 = int(up(C, 4) / 4);
  const bool two = q.w_dtype == DSF_BF16;
  const long long items = R * n4;
  float* u = reinterpret_cast<float*>(ws + w.u);
  float* squares = reinterpret_cast<float*>(ws + w.squares);
  const unsigned norm_blocks = blocks_for(items) < kNormBlocks ? blocks_for(items) : kNormBlocks;
  MomentArgs ma{q.g, q.m, u, squares, q.ldg, w.ldx, int(R), int(C), n4, false, at(q.m, 16) && C % 4 == 0, q.nesterov, q.mu};
  const int ges = q.g_dtype == DSF_F32 ? 4 : 2;
  ma.g_vec = at(q.g, 4 * ges) && q.ldg % 4 == 0;
  if (!pdl_launch(q.g_dtype == DSF_F32 ? moment_kernel<float> : moment_kernel<__nv_bfloat16>, dim3(norm_blocks), 256, s, ma))
    return false;
  __nv_bfloat16* x = reinterpret_cast<__nv_bfloat16*>(ws + w.x);
  if (!pdl_launch(scale_kernel, dim3(blocks_for(items)), 256, s,
                  ScaleArgs{u, squares, x, w.ldx, w.ldx, R * w.ldx, int(R), n4, int(norm_blocks), two}))
    return false;
  const long long n = w.n;
  const bool wide = R <= C;
  const long long terms = two ? 2 : 3;
  const Mat X{x, R, C, w.ldx, terms, R * w.ldx}, A{ws + w.a_terms, n, n, w.lda, terms, n * w.lda},
      B{ws + w.b_terms, n, n, w.lda, terms, n * w.lda};
  float* a32 = reinterpret_cast<float*>(ws + w.a);
  Product p;
  for (int i = 0; i < q.steps; ++i) {
    JoinArgs j{};
    j.f32 = a32;
    j.ldt = w.lda;
    j.tplane = n * w.lda;
    j.terms = reinterpret_cast<__nv_bfloat16*>(ws + w.a_terms);
    if (!part_product(p, two, wide ? kKK : kNN, X, X, n, n, wide ? C : R, ws, w, status, s) || !join<kSum, float>(p, j, ws, w, s))
      return false;
    j.terms = reinterpret_cast<__nv_bfloat16*>(ws + w.b_terms);
    if (!part_product(p, two, kKK, A, A, n, n, n, ws, w, status, s) || !join<kPoly, float>(p, j, ws, w, s)) return false;
    const bool ok = wide ? part_product(p, two, kKN, B, X, R, C, n, ws, w, status, s)
                         : part_product(p, two, kKK, X, B, R, C, n, ws, w, status, s);
    if (!ok) return false;
    JoinArgs f{};
    if (i + 1 < q.steps) {
      f.terms = x;
      f.ldt = w.ldx;
      f.tplane = R * w.ldx;
      if (!join<kSum, float>(p, f, ws, w, s)) return false;
      continue;
    }
    const int wes = q.w_dtype == DSF_F32 ? 4 : 2;
    f.W = q.W;
    f.ldw = q.ldw;
    f.w_vec = at(q.W, 4 * wes) && q.ldw % 4 == 0;
    f.decay = 1.f - q.lr * q.decay;
    f.rate = q.lr * (R > C ? sqrtf(float(R) / float(C)) : 1.f);
    return q.w_dtype == DSF_F32 ? join<kStep, float>(p, f, ws, w, s) : join<kStep, __nv_bfloat16>(p, f, ws, w, s);
  }
  return true;
}

bool muon_sizes_ok(int32_t R, int32_t C) { return R >= 1 && C >= 1 && R <= kMaxDim && C <= kMaxDim; }

}  // namespace
}  // namespace dense
}  // namespace dsf

using namespace dsf::dense;

extern "C" {

size_t dsf_muon_workspace_bytes(int32_t R, int32_t C) {
  if (!muon_sizes_ok(R, C) || (R < C ? R : C) > kMaxShort) return 0;
  return muon_layout(R, C).total;
}

int ctr_muon_update(void* W, int64_t ldw, int32_t w_dtype, const void* grad, int64_t ldg, int32_t g_dtype, float* momentum,
                    int32_t R, int32_t C, float lr, float mu, float weight_decay, int32_t nesterov, int32_t steps, void* ws,
                    size_t ws_bytes, int32_t* status, void* stream) {
  if ((w_dtype != DSF_F32 && w_dtype != DSF_BF16) || (g_dtype != DSF_F32 && g_dtype != DSF_BF16)) return DSF_EUNSUPPORTED;
  if (!muon_sizes_ok(R, C)) return DSF_EINVAL;
  if ((R < C ? R : C) > kMaxShort) return DSF_EUNSUPPORTED;
  const int wes = w_dtype == DSF_F32 ? 4 : 2, ges = g_dtype == DSF_F32 ? 4 : 2;
  if (!W || !at(W, wes) || ldw < C || !grad || !at(grad, ges) || ldg < C || !momentum || !at(momentum, 4)) return DSF_EINVAL;
  const bool finite = lr - lr == 0.f && weight_decay - weight_decay == 0.f;
  if (!finite || !(mu >= 0.f && mu < 1.f) || weight_decay < 0.f || nesterov < 0 || nesterov > 1 || steps < 1 ||
      steps > kMaxSteps)
    return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < muon_layout(R, C).total) return DSF_EWORKSPACE;
  const Step q{W, ldw, w_dtype, grad, ldg, g_dtype, momentum, lr, mu, weight_decay, nesterov != 0, steps};
  return muon(q, R, C, static_cast<uint8_t*>(ws), status, static_cast<cudaStream_t>(stream)) ? DSF_OK : DSF_ECUDA;
}

}  // extern "C"
