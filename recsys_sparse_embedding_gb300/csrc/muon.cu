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
// three bf16 terms each (six products of terms; X ends 5e-7 to 6e-6 off. The updated W
// is 1.0e-7 off, twice what products in fp32 leave: 512 x 256). A bf16 W is rounded to
// 2^-8 of an element at most in the end: two terms (2^-17, three products) leave X 2e-5
// to 6e-5 off, which W's rounding hides at half the work. (Of fewer than 64 rows or
// columns up to 4e-4: an error of a large singular value's direction grows with a small
// one's. One bf16 product would leave 1 to 3% of X, one fp16 0.2 to 0.3%.)
//
// A step's three products (2 n^2 m, 2 n^3 and 2 n^2 m operations; the first two are
// symmetric, and large ones are made by half) leave the next operand's terms in their
// epilogues; where a product is better split over K, it leaves fp32 partial sums that
// a second kernel adds up and lays out.
#include "dense_host.cuh"

namespace dsf {
namespace dense {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f, kEps = 1e-7f;
constexpr int kMaxShort = 1 << 15, kMaxSteps = 16;
constexpr int kNormBlocks = 512;
constexpr size_t kTriBytes = 2 * kPartBytes;  // of A's partial sums (whole squares, though half of the tiles are made)

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
// (kMirror, kMirrorPoly: kSum and kPoly by mirror_kernel)
enum { kSum = 0, kPoly = 1, kStep = 2, kMirror = 3, kMirrorPoly = 4 };
struct JoinArgs {
  const float* part;
  long long ldp, plane;
  int splits, M, N, n4;
  float* f32;  // [M][ld32]
  long long ld32;
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
      const float4 f = *reinterpret_cast<const float4*>(a.f32 + r * a.ld32 + c);
      const float A[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fmaf(kC, v[k], kB * A[k]) + (r == c + k ? kA : 0.f);
    } else if (a.f32) {
      *reinterpret_cast<float4*>(a.f32 + r * a.ld32 + c) = make_float4(v[0], v[1], v[2], v[3]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k >= n) v[k] = 0.f;
    put_terms(a.terms + r * a.ldt + c, a.tplane, v, a.two);
  }
}

// A symmetric product's partial sums, of which the lower triangle is there, as
// join_kernel's kSum or kPoly. A block has 32 x 32 elements of the triangle and writes them,
// turned over in shared memory, above the diagonal too.
template <bool POLY>
__global__ void __launch_bounds__(256) mirror_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float tile[32][33];
  pdl_go();
  pdl_wait();
  const int b = blockIdx.x, r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
  int i = int((sqrtf(8.f * float(b) + 1.f) - 1.f) * 0.5f);
  if (i * (i + 1) / 2 > b) --i;
  if ((i + 1) * (i + 2) / 2 <= b) ++i;
  const int r0 = i * 32, c0 = (b - i * (i + 1) / 2) * 32;
  auto out = [&](long long row, int col, float* v) {
    if (row >= a.N || col >= a.N) return;
    float4* q = reinterpret_cast<float4*>(a.f32 + row * a.ld32 + col);
    if (POLY) {
      const float4 f = *q;
      const float A[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fmaf(kC, v[k], kB * A[k]) + (row == col + k ? kA : 0.f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k >= a.N) v[k] = 0.f;
    if (!POLY) *q = make_float4(v[0], v[1], v[2], v[3]);
    put_terms(a.terms + row * a.ldt + col, a.tplane, v, a.two);
  };
  float v[4] = {};
  if (r0 + r < a.N && c0 + c < a.N) {
    const float* p = a.part + (long long)(r0 + r) * a.ldp + c0 + c;
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {
      const float4 f = *reinterpret_cast<const float4*>(p + z * a.plane);
      v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) tile[r][c + k] = v[k];
  out(r0 + r, c0 + c, v);
  __syncthreads();
  if (r0 == c0) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = tile[c + k][r];
  out(c0 + r, r0 + c, v);
}

struct MuonLayout {
  size_t x, x1, a_terms, b_terms, a, u, squares, part, total;
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
  auto part_of = [](size_t outputs, long long K, size_t room) {
    const size_t all = outputs * 4 * kMaxSplits, may = all < room ? all : room;
    const size_t least = outputs * 4 * size_t(least_splits_two((K + 63) / 64));
    return may > least ? may : least;
  };
  const size_t px = part_of(size_t(R) * w.ldx, w.n, kPartBytes), pa = part_of(size_t(w.n) * w.lda, R > C ? R : C, kTriBytes);
  w.x = take(size_t(R) * w.ldx * 6);
  w.x1 = take(size_t(R) * w.ldx * 6);
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

struct Operand {  // terms [.][rows][ld]
  __nv_bfloat16* p;
  long long rows, cols, ld;
  Mat mat(long long terms) const { return Mat{p, rows, cols, ld, terms, rows * ld}; }
};

struct Call {
  bool two;
  uint8_t* ws;
  MuonLayout w;
  int* status;
  cudaStream_t s;
};

// A B (or A B^T, A^T B by `major`) over K terms of the sum, planned.
Product planned(const Call& c, int major, const Operand& A, const Operand& B, long long M, long long N, long long K, bool split,
                double* time) {
  Product p{};
  p.major = major;
  p.f32 = !c.two;
  p.two = c.two;
  p.epi = kEpiOut;
  *time = plan(p, M, N, 1, (K + 63) / 64, 1, split);
  if (p.a.job[0].splits == 1) *time += split ? Cost::kSecond : 0;  // (its second launch, if it leaves sums)
  p.A = A.mat(c.two ? 2 : 3);
  p.B = B.mat(c.two ? 2 : 3);
  p.a.status = c.status;
  p.a.job[0].a_term = p.a.job[0].b_term = 1;
  return p;
}

// The product's partial sums to w.part, then the join.
template <int MODE, class TW>
bool split_product(const Call& c, Product p, JoinArgs j) {
  Job& o = p.a.job[0];
  p.epi = kEpiPart;
  o.out = c.ws + c.w.part;
  o.ldo = up(o.N, 4);
  o.out_plane = o.M * o.ldo;
  o.out_vec = 1;
  if (!(c.two ? run_two_product(p, c.s) : (p.major == kKK ? run_fwd_product(p, c.s) : run_grad_product(p, c.s)))) return false;
  j.part = reinterpret_cast<const float*>(c.ws + c.w.part);
  j.ldp = o.ldo;
  j.plane = o.out_plane;
  j.splits = o.splits;
  j.M = o.M;
  j.N = o.N;
  j.n4 = int(o.ldo / 4);
  j.two = c.two;
  if constexpr (MODE >= kMirror) {
    const long long b = (j.N + 31) / 32;
    return pdl_launch(mirror_kernel<MODE == kMirrorPoly>, dim3(unsigned(b * (b + 1) / 2)), 256, c.s, j);
  } else {
    return pdl_launch(join_kernel<MODE, TW>, dim3(blocks_for((long long)j.M * j.n4)), 256, c.s, j);
  }
}

// Up to this size of the output three terms are written faster by the second kernel than
// by a product's epilogue, one item of a warp after the other, by 3 us or so. (Calls of
// 64 x 64 88 and 73 us, 256 x 256 139 and 117, 300 x 900 153 and 136; but if larger outputs
// are split too, 8192 x 512 285 and 308, 20,000 x 300 411 and 431; in two terms 64 x 64 62
// and 66.)
constexpr long long kSmallOutput = 300000;

// The product to out's terms (and fp32 f32 [M][out.ld], nullable), or, with poly, those
// of the polynomial with A = f32.
bool terms_product(const Call& c, int major, const Operand& A, const Operand& B, long long K, const Operand& out, float* f32,
                   bool poly) {
  double whole, parts;
  Product p = planned(c, major, A, B, out.rows, out.cols, K, false, &whole);
  const Product q = planned(c, major, A, B, out.rows, out.cols, K, true, &parts);
  const double ahead = !c.two && out.rows * out.cols <= kSmallOutput ? 3 : 0;
  if (whole <= parts - ahead && (!c.two || least_splits_two((K + 63) / 64) == 1)) {
    Job& o = p.a.job[0];
    p.epi = poly ? kEpiPoly : kEpiTerms;
    o.out = out.p;
    o.ldo = out.ld;
    o.out_plane = out.rows * out.ld;
    o.out_vec = 1;
    if (poly) {
      p.a.in = f32;
      p.a.ldi = out.ld;
      p.a.in_vec = 1;
      p.a.c0 = kA, p.a.c1 = kB, p.a.c2 = kC;
    } else {
      p.a.f32 = f32;
    }
    return run_terms_product(p, c.s);
  }
  JoinArgs j{};
  j.f32 = f32;
  j.ld32 = out.ld;
  j.terms = out.p;
  j.ldt = out.ld;
  j.tplane = out.rows * out.ld;
  return poly ? split_product<kPoly, float>(c, q, j) : split_product<kSum, float>(c, q, j);
}

// The symmetric products: A = X X^T (or X^T X) over K terms of the sum, or the polynomial
// in A from A A. From n = 1024 on only the tiles of the lower triangle are made, added up
// and mirrored, the polynomial's where that is faster than its own epilogue. (A with all of
// its tiles and with these, the call's us: fp32 1024 x 4096 460 and 421, 4096 x 4096 7337
// and 6371; bf16 8192 x 1024 454 and 411; but fp32 512 x 256 121 and 130, bf16 20,000 x
// 300 320 and 367, 700 x 900 172 and 175: few blocks then add up many splits.
// The polynomial: fp32 1024 x 4096 421 and 402, 4096 x 4096 6371 and 5513.)
constexpr long long kMirrorFrom = 1024;
bool symmetric_product(const Call& c, int major, const Operand& X, long long K, const Operand& out, float* a32, bool poly) {
  const long long n = out.rows;
  if (n < kMirrorFrom) return terms_product(c, major, X, X, K, out, a32, poly);
  double whole, parts;
  planned(c, major, X, X, n, n, K, false, &whole);
  Product p = planned(c, major, X, X, n, n, K, true, &parts);
  const double time = plan_tri(p, n, (K + 63) / 64, kTriBytes);
  if (poly && whole <= time) return terms_product(c, major, X, X, K, out, a32, poly);
  JoinArgs j{};
  j.f32 = a32;
  j.ld32 = out.ld;
  j.terms = out.p;
  j.ldt = out.ld;
  j.tplane = n * out.ld;
  return poly ? split_product<kMirrorPoly, float>(c, p, j) : split_product<kMirror, float>(c, p, j);
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
  auto at_ws = [&](size_t o) { return reinterpret_cast<__nv_bfloat16*>(ws + o); };
  const Call c{two, ws, w, status, s};
  const Operand A{at_ws(w.a_terms), n, n, w.lda}, B{at_ws(w.b_terms), n, n, w.lda};
  Operand X{x, R, C, w.ldx}, Y{at_ws(w.x1), R, C, w.ldx};
  float* a32 = reinterpret_cast<float*>(ws + w.a);
  for (int i = 0; i < q.steps; ++i) {
    if (!symmetric_product(c, wide ? kKK : kNN, X, wide ? C : R, A, a32, false) || !symmetric_product(c, kKK, A, n, B, a32, true))
      return false;
    const int major = wide ? kKN : kKK;
    const Operand &left = wide ? B : X, &right = wide ? X : B;
    if (i + 1 < q.steps) {
      if (!terms_product(c, major, left, right, n, Y, nullptr, false)) return false;
      const Operand t = X;
      X = Y;
      Y = t;
      continue;
    }
    double time;
    const Product p = planned(c, major, left, right, R, C, n, true, &time);
    JoinArgs f{};
    const int wes = q.w_dtype == DSF_F32 ? 4 : 2;
    f.W = q.W;
    f.ldw = q.ldw;
    f.w_vec = at(q.W, 4 * wes) && q.ldw % 4 == 0;
    f.decay = 1.f - q.lr * q.decay;
    f.rate = q.lr * (R > C ? sqrtf(float(R) / float(C)) : 1.f);
    return q.w_dtype == DSF_F32 ? split_product<kStep, float>(c, p, f) : split_product<kStep, __nv_bfloat16>(c, p, f);
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
