// The dense operators of any width (declared in dinsparse.h): argument checks,
// workspace layout and the kernels' launches.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "colsum.cuh"
#include "dense_small.cuh"
#include "dense_tc.cuh"
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

// ---------------------------------------------------------------- the products' shapes
constexpr int kSms = 152;
constexpr int kMaxSplits = 32;
// partial sums of a split product: units fill the chip at most once, and a
// unit holds at most 256 x 256 fp32 per pair of SMs
constexpr size_t kPartBytes = size_t(kSms / 2) * 256 * 256 * 4;

// Estimates in microseconds, per tile configuration (fitted to measured calls
// of 200 to 8192 rows; checked on 26 shapes of 64 to 8192 rows, the pick is
// within 5% of the best of the three but for the gated forward of 8192 x 256 ->
// 684, 19.0 us against 16.0): a K-block of a 256 x 256 tile (on two SMs; fp32: 256 x
// 128, six products), 128 x 128, 128 x 64 or (in runs) 256 x 128 tile takes `block`, its epilogue
// `tail`, and the two overlap from tile to tile; a launch costs kLaunch; the
// chip takes its units in whole waves; a split product pays for a second
// launch and its partial sums' way to L2 and back.
struct Cost {
  bool f32;
  double block(int cfg) const {
    constexpr double kBlock[2][4] = {{0.31, 0.29, 0.275, 0.23}, {0.9, 0.95, 0.75, 0}};
    return kBlock[f32][cfg];
  }
  double tail(int cfg) const {
    constexpr double kTail[2][4] = {{4.4, 2.2, 1.2, 2.6}, {3.0, 3.0, 2.0, 0}};
    return kTail[f32][cfg];
  }
  // `units` in a row, of `blocks` K-blocks each
  double run(int cfg, double units, double blocks) const {
    const double m = blocks * block(cfg), e = tail(cfg);
    return units * (m > e ? m : e) + (m > e ? e : m);
  }
  static constexpr double kLaunch = 2.4, kSecond = 2.2, kBytesPerUs = 4e6;
  static double parts(long long splits, double outputs) {
    return splits > 1 ? kSecond + double(splits) * outputs * 8 / kBytesPerUs : 0;
  }
};

// The tiles of a product [nb][M][N] over segments of nkb K-blocks.
void set_tiles(Job& o, int cfg, long long M, long long N, int nb, bool gated, bool f32, long long nkb, int nseg,
               long long want) {
  const long long on = cfg_bn(cfg, f32) / (gated ? 2 : 1), rows = cfg_rows(cfg);
  o.M = int(M);
  o.N = int(N);
  o.mt = int((M + rows - 1) / rows);
  o.nt = int((N + on - 1) / on);
  o.nb = nb;
  o.nkb = int(nkb);
  o.kbps = int((nkb + want - 1) / want);
  o.splits = int((nkb + o.kbps - 1) / o.kbps);
  o.nseg = nseg;
}
long long tiles_of(const Job& o) { return (long long)o.mt * o.nt * o.nb; }
long long slots_of(int cfg) { return kSms * 128 / cfg_rows(cfg); }

// K-blocks that a bf16 or e4m3 product takes in one accumulator run at most (as
// far as kMaxSplits go): longer sums are split, and their parts added in fp32. A
// sum of n = 4 kLongRun additions that truncate is low by up to 3 n 2^-25 =
// 3.7e-4 of itself, a tenth of a bf16 rounding; over 2^20 inputs it would be 6e-3.
constexpr long long kLongRun = 1024;

// Splits that a product of `blocks` K-blocks has at least.
long long least_splits(bool f32, long long blocks) {
  const long long n = (blocks + kLongRun - 1) / kLongRun;
  return f32 || n < 1 ? 1 : (n < kMaxSplits ? n : kMaxSplits);
}

// K-blocks in one accumulator run of a bf16 dz product that db is summed from.
// With more, its wide tiles are half as wide (configuration 3), so that the
// epilogue's registers hold a tile's sums. (Without db, dz is rounded to bf16,
// and the runs would not be seen.)
constexpr long long kDzBlocks = 8;

// Picks the configuration and the K-splits of one product.
void plan(Product& p, long long M, long long N, int nb, long long nkb, int nseg, bool may_split) {
  const Cost cost{p.f32};
  double best = 1e300;
  Job o = p.a.job[0];
  const bool runs = p.epi == kEpiDz && !p.f32 && nkb > (p.a.part ? kDzBlocks : kLongRun);
  const long long least = may_split ? least_splits(p.f32, nkb * nseg) : 1;
  for (int cfg = 0; cfg < 4; ++cfg) {
    if (cfg == 2 && p.gated) continue;
    if (cfg % 3 == 0 && (cfg == 3) != runs) continue;
    for (long long want = least; want <= kMaxSplits && want <= nkb; ++want) {
      set_tiles(o, cfg, M, N, nb, p.gated, p.f32, nkb, nseg, want);
      if (tiles_of(o) > INT32_MAX / 64) break;
      if (want > least && (!may_split || tiles_of(o) * want > slots_of(cfg))) break;
      if (want > least && o.splits != want) continue;
      const long long waves = (tiles_of(o) * o.splits + slots_of(cfg) - 1) / slots_of(cfg);
      const double c = Cost::kLaunch + cost.run(cfg, double(waves), double(o.kbps) * nseg) +
                       Cost::parts(o.splits, double(M) * N * nb * (p.gated ? 2 : 1));
      if (c < best) {
        best = c;
        p.cfg = cfg;
        p.a.job[0] = o;
      }
    }
  }
}

// dW (job 0, which may be split) and dx (job 1) in one launch.
void plan_dual(Product& p, long long M, long long N, long long K, int halves) {
  const Cost cost{p.f32};
  const long long kw = (M + 63) / 64, kx = (N + 63) / 64, least = least_splits(p.f32, kw);
  double best = 1e300;
  TcArgs a = p.a;
  for (int cfg = 0; cfg < 3; ++cfg)
    for (long long want = least; want <= kMaxSplits && want <= kw; ++want) {
      set_tiles(a.job[0], cfg, N, K, halves, false, p.f32, kw, 1, want);
      set_tiles(a.job[1], cfg, M, K, 1, false, p.f32, kx, halves, 1);
      const Job& w = a.job[0];
      if (tiles_of(w) > INT32_MAX / 64 || tiles_of(a.job[1]) > INT32_MAX / 64) break;
      if (want > least && tiles_of(w) * want > slots_of(cfg)) break;
      if (want > least && w.splits != want) continue;
      const double tail = cost.tail(cfg), tw = w.kbps * cost.block(cfg), tx = double(kx) * halves * cost.block(cfg);
      const long long weight[2] = {(long long)(1e3 * (tw > tail ? tw : tail)), (long long)(1e3 * (tx > tail ? tx : tail))};
      const Deal d = deal(a, weight, slots_of(cfg));
      const double c = Cost::kLaunch + 1e-3 * double(d.load) + tail + Cost::parts(w.splits, double(N) * K * halves);
      if (c < best) {
        best = c;
        p.cfg = cfg;
        p.a.job[0] = a.job[0];
        p.a.job[1] = a.job[1];
        p.weight[0] = weight[0];
        p.weight[1] = weight[1];
      }
    }
}

long long up(long long v, long long to) { return (v + to - 1) / to * to; }

// Workspace layout of a call: each part's offset; `total` grows with M.
struct Layout {
  size_t xp, wp, gp, dz, sums, part, total;
  long long kp, np;  // padded row lengths of the laid-out operands and of dz
};

// Whether an operand with rows of `cols` elements is laid out in the workspace.
bool laid_out(int dtype, long long cols) { return dtype == DSF_F32 || (cols * esize(dtype)) % 16 != 0; }

Layout layout(const dsf_dense* l, long long M, bool gated, bool backward) {
  Layout w{};
  const int es = esize(l->dtype), terms = l->dtype == DSF_F32 ? 3 : 1, pes = l->dtype == DSF_F32 ? 2 : es;
  const long long N = gated ? l->R / 2 : l->R, halves = gated ? 2 : 1;
  w.kp = up(l->K, 16 / pes);
  w.np = up(N, 8);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  // partial sums of a product of `blocks` K-blocks: those of the splits that it
  // may have, or of those that it has at least
  auto part_of = [l](size_t outputs, long long blocks) {
    const size_t b = outputs * 4 * kMaxSplits, may = b < kPartBytes ? b : kPartBytes;
    const size_t least = size_t(least_splits(l->dtype == DSF_F32, blocks));
    return least > 1 && outputs * 4 * least > may ? outputs * 4 * least : may;
  };
  auto blocks_of = [](long long k, int per) { return (k + per - 1) / per; };
  const bool lo = laid_out(l->dtype, l->K);
  w.xp = take(lo ? size_t(terms) * M * w.kp * pes : 0);
  w.wp = take(lo ? size_t(terms) * l->R * w.kp * pes : 0);
  size_t part = part_of(size_t(M) * up(N, 4) * halves, blocks_of(l->K, l->dtype == DSF_E4M3 ? 128 : 64));
  if (backward) {
    const bool own_dz = gated || l->act != DSF_ACT_NONE;  // else dz is dy
    w.gp = take(!own_dz && laid_out(l->dtype, N) ? size_t(terms) * M * w.np * pes : 0);
    w.dz = take(own_dz ? size_t(terms) * halves * M * w.np * 2 : 0);
    w.sums = take(size_t((M + 31) / 32) * l->R * 4);
    const size_t px = part_of(size_t(M) * up(l->K, 4), blocks_of(N, 64) * halves);
    const size_t pw = part_of(size_t(l->R) * up(l->K, 4), blocks_of(M, 64));
    part = part > px ? part : px;
    part = part > pw ? part : pw;
  }
  w.part = take(part);
  w.total = o + 256;
  return w;
}

size_t ws_bytes_of(const dsf_dense* l, long long M, bool gated, bool backward) {
  return layout(l, M, gated, backward).total;
}

// ---------------------------------------------------------------- small kernels
// Lays a matrix out for the products: rows of `cols` elements from src (row
// stride ld) into rows of ldd. fp32: the three bf16 terms, plane t at t *
// rows * ldd; otherwise a copy. One thread per 8 (16-bit) or 16 (8-bit)
// elements of a destination row.
struct LayJob {
  const void* src;
  void* dst;
  long long ld, rows, ldd, cols;
};
struct LayJobs {
  LayJob j[3];
  int b0, b1;  // blocks [0, b0) take job 0, [b0, b1) job 1, the others job 2
};

// The n (2 or 3) 16-byte vectors that hold the bytes from p on, shifted so that
// w[0] starts with p's: bytes [p, p + 16 (n - 1)). p is a multiple of ES.
template <int NV, int ES>
__device__ __forceinline__ void load_shifted(const uint8_t* p, uint32_t* w) {
  const uint32_t o = uint32_t(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* q = reinterpret_cast<const uint4*>(p - o);
  uint32_t v[4 * NV + 4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint4 x = __ldg(q + i);
    v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 * NV + i] = 0;
  if (o & 8u) {
#pragma unroll
    for (int i = 0; i < 4 * NV - 2; ++i) v[i] = v[i + 2];
  }
  if (o & 4u) {
#pragma unroll
    for (int i = 0; i < 4 * NV - 2; ++i) v[i] = v[i + 1];
  }
#pragma unroll
  for (int i = 0; i < 4 * (NV - 1); ++i) w[i] = ES == 4 ? v[i] : __funnelshift_r(v[i], v[i + 1], (o & 3u) * 8u);
}

template <int ES>  // source element: 4 (fp32 -> three bf16 terms), 2 or 1 (copied)
__global__ void __launch_bounds__(256) lay_kernel(const __grid_constant__ LayJobs a) {
  pdl_go();
  pdl_wait();
  const int blk = int(blockIdx.x), which = blk < a.b0 ? 0 : (blk < a.b1 ? 1 : 2);
  const LayJob& j = a.j[which];  // (indexed in place: a choice among parameters would be copied to the stack)
  const int first = which == 0 ? 0 : (which == 1 ? a.b0 : a.b1);
  const int nblk = (which == 0 ? a.b0 : (which == 1 ? a.b1 : int(gridDim.x))) - first, local = blk - first;
  constexpr int V = ES == 1 ? 16 : 8, NW = V * ES / 4, NV = NW / 4 + 1;  // elements, words, vectors of a piece
  // a block takes whole rows side by side, or parts of one
  const int per_row = int(j.ldd / V), tpr = min(per_row, 256), rpb = 256 / tpr;
  const int rr = int(threadIdx.x) / tpr, c0 = int(threadIdx.x) - rr * tpr;
  if (rr >= rpb) return;
  const uint8_t* end = static_cast<const uint8_t*>(j.src) + ((j.rows - 1) * j.ld + j.cols) * ES;
  for (long long r = (long long)local * rpb + rr; r < j.rows; r += (long long)nblk * rpb)
   for (int c = c0 * V; c < j.ldd; c += tpr * V) {
    const uint8_t* s = static_cast<const uint8_t*>(j.src) + (r * j.ld + c) * ES;
    uint32_t w[NW];
    // (whole vectors where all of them lie inside the matrix; what a row's last
    // piece takes from behind the row is never read)
    if (s - 15 >= static_cast<const uint8_t*>(j.src) && s + 16 * NV <= end) {
      load_shifted<NV, ES>(s, w);
    } else {
#pragma unroll
      for (int k = 0; k < NW; ++k) w[k] = 0;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (c + k >= j.cols) continue;
        if (ES == 4) w[k * ES / 4] = reinterpret_cast<const uint32_t*>(s)[k];
        if (ES == 2) w[k * ES / 4] |= uint32_t(reinterpret_cast<const uint16_t*>(s)[k]) << (16 * (k % 2));
        if (ES == 1) w[k * ES / 4] |= uint32_t(s[k]) << (8 * (k % 4));
      }
    }
    if constexpr (ES == 4) {
      uint16_t* d = static_cast<uint16_t*>(j.dst) + r * j.ldd + c;
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = take_term(x[2 * k]), hi = take_term(x[2 * k + 1]);
          h[k] = __byte_perm(lo, hi, 0x7632);
        }
        *reinterpret_cast<uint4*>(d + t * j.rows * j.ldd) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(j.dst) + (r * j.ldd + c) * ES) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

bool lay(int dtype, const LayJob* jobs, int n, cudaStream_t s) {
  LayJobs a{};
  int b[3] = {}, tot = 0;
  const int V = dtype == DSF_E4M3 ? 16 : 8;
  for (int i = 0; i < n; ++i) {
    a.j[i] = jobs[i];
    const long long per_row = jobs[i].ldd / V, rpb = per_row < 256 ? 256 / per_row : 1;
    const long long blocks = (jobs[i].rows + rpb - 1) / rpb;
    b[i] = int(blocks < kSms * 16 ? blocks : kSms * 16);
    tot += b[i];
  }
  if (tot == 0) return true;
  auto* kernel = dtype == DSF_F32 ? lay_kernel<4> : (dtype == DSF_BF16 ? lay_kernel<2> : lay_kernel<1>);
  a.b0 = b[0];
  a.b1 = b[0] + b[1];
  return pdl_launch(kernel, dim3(unsigned(tot)), 256, s, a);
}

// Sums over blocks of 32 rows of a matrix (db where dz is dy): part[block][n].
// VEC: 16 bytes of a row per lane; else one element. (8192 x 1024 in bf16 with
// the sum over blocks: 5.1 us; 6.5 with 64 rows, 7.7 with 128.)
constexpr int kSumRows = 32;
template <class T, bool VEC>
__global__ void __launch_bounds__(256) row_block_sums_kernel(const T* g, long long ld, long long M, int N, float* part) {
  constexpr int E = VEC ? 16 / int(sizeof(T)) : 1;
  __shared__ float p[8][32 * E];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n0 = blockIdx.y * 32 * E;
  const int n = n0 + lane * E;  // (VEC: rows are whole vectors, what they hold past N is not stored)
  const long long r0 = (long long)blockIdx.x * kSumRows;
  pdl_go();
  pdl_wait();
  float s[E] = {};
  if (n < N) {
    constexpr int U = 4;  // rows in flight
#pragma unroll 1
    for (int i0 = 0; i0 < kSumRows / 8; i0 += U) {
      const T* q = g + (r0 + w + 8 * i0) * ld + n;
      if constexpr (VEC) {
        uint4 u[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
          u[i] = r0 + w + 8 * (i0 + i) < M ? __ldg(reinterpret_cast<const uint4*>(q + 8 * i * ld)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float v[E];
          unpack(u[i], v, T());
#pragma unroll
          for (int e = 0; e < E; ++e) s[e] += v[e];
        }
      } else {
        float v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = r0 + w + 8 * (i0 + i) < M ? elem(q[8 * i * ld]) : 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) s[0] += v[i];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) p[w][lane * E + e] = s[e];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * E; c += 256) {
    if (n0 + c >= N) break;
    float v = p[0][c];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += p[k][c];
    part[(long long)blockIdx.x * N + n0 + c] = v;
  }
}
template <class T>
bool row_block_sums(const void* g, long long ld, bool padded, long long M, int N, float* part, cudaStream_t s) {
  constexpr int E = 16 / int(sizeof(T));
  const T* q = static_cast<const T*>(g);
  const unsigned blocks = unsigned((M + kSumRows - 1) / kSumRows);
  if (at(g, 16) && (ld * int(sizeof(T))) % 16 == 0 && (N % E == 0 || padded))
    return pdl_launch(row_block_sums_kernel<T, true>, dim3(blocks, unsigned((N + 32 * E - 1) / (32 * E))), 256, s, q, ld, M,
                      N, part);
  return pdl_launch(row_block_sums_kernel<T, false>, dim3(blocks, unsigned((N + 31) / 32)), 256, s, q, ld, M, N, part);
}

// The end of a split product: the splits' partial sums, added in order, then
// the forward's epilogue (fwd) or the plain sum. Four columns per thread.
struct FinishArgs {
  const float* part;  // [splits][planes][M][ldp]
  long long M, ldp;
  int N, splits, planes;
  bool fwd, gated;
  const float *bias, *xs, *ws;
  const void* res;
  long long ldr;
  void* out;
  long long ldo, out_plane;
  int act;
};
template <class TO>
__global__ void __launch_bounds__(256) finish_kernel(const FinishArgs a) {
  pdl_go();
  pdl_wait();
  const long long n4 = a.ldp / 4, per = a.M * n4, plane = a.M * a.ldp;
  const long long total = per * (a.gated ? 1 : a.planes);
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long b = i / per, r = i - b * per, m = r / n4;
    const int n = int(r - m * n4) * 4;
    float v[2][4] = {};
    const float* p = a.part + b * plane + m * a.ldp + n;
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {
      const float* q = p + (long long)z * a.planes * plane;
      const float4 f = *reinterpret_cast<const float4*>(q);
      v[0][0] += f.x, v[0][1] += f.y, v[0][2] += f.z, v[0][3] += f.w;
      if (a.gated) {
        const float4 h = *reinterpret_cast<const float4*>(q + plane);
        v[1][0] += h.x, v[1][1] += h.y, v[1][2] += h.z, v[1][3] += h.w;
      }
    }
    TO* o = static_cast<TO*>(a.out) + b * a.out_plane + m * a.ldo + n;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (n + k >= a.N) break;
      float z = v[0][k];
      if (a.fwd) {
        if (a.xs) z *= a.xs[m] * a.ws[n + k];
        if (a.bias) z += a.bias[n + k];
        z = act_any(a.act, z);
        if (a.gated) {
          float u = v[1][k];
          if (a.xs) u *= a.xs[m] * a.ws[a.N + n + k];
          if (a.bias) u += a.bias[a.N + n + k];
          z *= u;
        }
        if (a.res) z += elem(static_cast<const TO*>(a.res)[m * a.ldr + n + k]);
      }
      o[k] = TO(z);
    }
  }
}

// ---------------------------------------------------------------- products
bool vec_rows(const void* p, long long ld, int es) { return at(p, 16) && (ld * es) % 16 == 0; }

struct Ctx {
  const dsf_dense* l;
  bool gated;
  long long M;
  int N, halves, es, eo, terms, kbe;  // kbe: K elements per K-block
  uint8_t* ws;
  Layout w;
  int* status;
  cudaStream_t s;
  Mat X, W;  // operands [terms][M][K], [terms * halves][N][K]
};

Ctx context(const dsf_dense* l, bool gated, const void* x, long long ldx, long long M, void* ws, bool backward,
            int* status, cudaStream_t s) {
  Ctx c{};
  c.l = l;
  c.gated = gated;
  c.M = M;
  c.halves = gated ? 2 : 1;
  c.N = l->R / c.halves;
  c.es = esize(l->dtype);
  c.eo = osize(l->dtype);
  c.terms = l->dtype == DSF_F32 ? 3 : 1;
  c.kbe = l->dtype == DSF_E4M3 ? 128 : 64;
  c.ws = static_cast<uint8_t*>(ws);
  c.w = layout(l, M, gated, backward);
  c.status = status;
  c.s = s;
  if (laid_out(l->dtype, l->K)) {
    c.X = Mat{c.ws + c.w.xp, M, l->K, c.w.kp, c.terms, M * c.w.kp};
    c.W = Mat{c.ws + c.w.wp, c.N, l->K, c.w.kp, (long long)c.terms * c.halves, c.N * c.w.kp};
  } else {
    c.X = Mat{x, M, l->K, ldx, 1, 0};
    c.W = Mat{l->W, c.N, l->K, l->ldw, c.halves, c.N * l->ldw};
  }
  return c;
}

bool lay_operands(const Ctx& c, const void* x, long long ldx, const void* dy, long long lddy) {
  LayJob jobs[3];
  int n = 0;
  if (laid_out(c.l->dtype, c.l->K)) {
    jobs[n++] = LayJob{x, c.ws + c.w.xp, ldx, c.M, c.w.kp, c.l->K};
    jobs[n++] = LayJob{c.l->W, c.ws + c.w.wp, c.l->ldw, c.l->R, c.w.kp, c.l->K};
  }
  if (dy && laid_out(c.l->dtype, c.N)) jobs[n++] = LayJob{dy, c.ws + c.w.gp, lddy, c.M, c.w.np, c.N};
  return lay(c.l->dtype, jobs, n, c.s);
}

// Job 0's partial sums.
void set_part(Product& p, const Ctx& c) {
  Job& o = p.a.job[0];
  p.epi = kEpiPart;
  o.out = c.ws + c.w.part;
  o.ldo = up(o.N, 4);
  o.out_plane = o.M * o.ldo;
  o.out_vec = 1;
}

void set_out(Job& o, void* out, long long ldo, int es) {
  o.out = out;
  o.ldo = ldo;
  o.out_plane = o.M * ldo;
  o.out_vec = vec_rows(out, ldo, es) && (o.nb == 1 || (o.out_plane * es) % 16 == 0);
}

bool finish(const Ctx& c, const Product& p, FinishArgs f, bool f32) {
  f.part = reinterpret_cast<const float*>(c.ws + c.w.part);
  const Job& o = p.a.job[0];
  f.M = o.M;
  f.N = o.N;
  f.ldp = o.ldo;
  f.splits = o.splits;
  const long long total = f.M * (f.ldp / 4) * (f.gated ? 1 : f.planes), blocks = (total + 255) / 256;
  const unsigned grid = unsigned(blocks < kSms * 16 ? blocks : kSms * 16);
  return pdl_launch(f32 ? finish_kernel<float> : finish_kernel<__nv_bfloat16>, dim3(grid), 256, c.s, f);
}

// x W^T with the forward's epilogue (dz null) or the backward's into dz.
bool layer_product(const Ctx& c, const float* xs, const void* in, long long ldi, void* y, long long ldy, bool dz,
                   float* sums) {
  const dsf_dense* l = c.l;
  const bool f32 = l->dtype == DSF_F32;
  Product p{};
  p.A = c.X;
  p.B = c.W;
  p.major = kKK;
  p.gated = c.gated;
  p.f32 = f32;
  p.epi = dz ? kEpiDz : (in ? kEpiRes : kEpiFwd);
  const long long nkb = (l->K + c.kbe - 1) / c.kbe;
  p.a.part = sums;
  plan(p, c.M, c.N, 1, nkb, 1, !dz);
  Job& o = p.a.job[0];
  o.a_term = 1;
  o.b_term = 1;
  p.a.act = l->act;
  p.a.bias = l->bias;
  p.a.xs = xs;
  p.a.ws = l->scale;
  p.a.status = c.status;
  if (o.splits > 1) {
    set_part(p, c);
  } else {
    p.a.in = in;
    p.a.ldi = ldi;
    p.a.in_vec = in && vec_rows(in, ldi, c.eo);
    set_out(o, y, ldy, dz ? 2 : c.eo);
  }
  const bool ok = dz ? run_dz_product(p, c.s) : (l->dtype == DSF_E4M3 ? run_e4m3_product(p, c.s) : run_fwd_product(p, c.s));
  if (!ok || o.splits == 1) return ok;
  FinishArgs f{};
  f.fwd = true;
  f.gated = c.gated;
  f.planes = c.halves;
  f.bias = l->bias;
  f.xs = xs;
  f.ws = l->scale;
  f.res = in;
  f.ldr = ldi;
  f.out = y;
  f.ldo = ldy;
  f.act = l->act;
  return finish(c, p, f, f32);
}

// The gradient products: dx (dz [.][M][N] times W) and dW (dz^T times x, one
// batch per half), each where asked for.
bool grad_products(const Ctx& c, const Mat& dz, void* dx, long long lddx, void* dW) {
  const int K = c.l->K;
  const bool f32 = c.l->dtype == DSF_F32;
  if (!dx && !dW) return true;
  // (in the launch for both, dx's sums are not split)
  if (dx && dW && least_splits(f32, (c.N + 63) / 64 * c.halves) > 1)
    return grad_products(c, dz, nullptr, 0, dW) && grad_products(c, dz, dx, lddx, nullptr);
  Product p{};
  p.gated = false;
  p.f32 = f32;
  p.epi = kEpiOut;
  p.a.status = c.status;
  if (dx && dW) {
    p.major = kDual;
    plan_dual(p, c.M, c.N, K, c.halves);
  } else {
    p.major = dW ? kNN : kKN;
    plan(p, dW ? c.N : c.M, K, dW ? c.halves : 1, ((dW ? c.M : c.N) + 63) / 64, dW ? 1 : c.halves, true);
  }
  Job &w = p.a.job[0], &x = p.a.job[dW ? 1 : 0];
  if (dW) {
    p.A = dz;
    p.B = c.X;
    w.a_term = c.halves;
    w.a_seg = 0;
    w.b_term = 1;
    set_out(w, dW, K, c.es);
  }
  if (dx) {
    (dW ? p.A1 : p.A) = dz;
    (dW ? p.B1 : p.B) = c.W;
    x.a_term = c.halves;
    x.a_seg = 1;
    x.b_term = c.halves;
    set_out(x, dx, lddx, c.es);
  }
  const Job out = p.a.job[0];
  if (out.splits > 1) set_part(p, c);
  if (!(dx && dW ? run_dual_product(p, c.s) : run_grad_product(p, c.s))) return false;
  if (out.splits == 1) return true;
  FinishArgs f{};
  f.planes = out.nb;
  f.out = out.out;
  f.ldo = out.ldo;
  f.out_plane = out.out_plane;
  return finish(c, p, f, f32);
}

int fwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const float* xs, const void* res, long long ldr,
        long long M, void* y, long long ldy, void* ws, int* status, cudaStream_t s) {
  bool ok;
  if (small_call(l->dtype, M, l->R, l->K)) {
    const int N = gated ? l->R / 2 : l->R;
    const SmallArgs a{x, l->W, ldx, l->ldw, l->bias, xs, l->scale, res, ldr, y, ldy, int(M), N, l->K, l->act, 0};
    const bool vec = (l->K * esize(l->dtype)) % 16 == 0;
    ok = l->dtype == DSF_F32    ? launch_small<float, float>(a, gated, vec, s)
         : l->dtype == DSF_BF16 ? launch_small<__nv_bfloat16, __nv_bfloat16>(a, gated, vec, s)
                                : launch_small<__nv_fp8_e4m3, __nv_bfloat16>(a, gated, vec, s);
  } else {
    const Ctx c = context(l, gated, x, ldx, M, ws, false, status, s);
    ok = lay_operands(c, x, ldx, nullptr, 0) && layer_product(c, xs, res, ldr, y, ldy, false, nullptr);
  }
  return ok ? DSF_OK : DSF_ECUDA;
}

int bwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const void* dy, long long lddy, long long M,
        void* dx, long long lddx, void* dW, float* db, void* ws, int* status, cudaStream_t s) {
  const Ctx c = context(l, gated, x, ldx, M, ws, true, status, s);
  const bool f32 = l->dtype == DSF_F32, own_dz = gated || l->act != DSF_ACT_NONE;
  float* sums = reinterpret_cast<float*>(c.ws + c.w.sums);
  if (!dx && !dW && !db) return DSF_OK;
  if ((own_dz || dx || dW) && !lay_operands(c, x, ldx, own_dz ? nullptr : dy, lddy)) return DSF_ECUDA;
  Mat dz;
  if (own_dz) {
    void* d = c.ws + c.w.dz;
    if (!layer_product(c, nullptr, dy, lddy, d, c.w.np, true, db ? sums : nullptr)) return DSF_ECUDA;
    if (db && !colsum(sums, (M + 31) / 32, l->R, db, s)) return DSF_ECUDA;
    dz = Mat{d, M, c.N, c.w.np, (long long)c.terms * c.halves, M * c.w.np};
  } else {
    if (db) {
      const long long blocks = (M + kSumRows - 1) / kSumRows;
      const bool laid = !f32 && laid_out(l->dtype, c.N) && (dx || dW);  // (the aligned copy of dy)
      const bool ok = f32    ? row_block_sums<float>(dy, lddy, false, M, c.N, sums, s)
                      : laid ? row_block_sums<__nv_bfloat16>(c.ws + c.w.gp, c.w.np, true, M, c.N, sums, s)
                             : row_block_sums<__nv_bfloat16>(dy, lddy, false, M, c.N, sums, s);
      if (!ok || !colsum(sums, blocks, c.N, db, s)) return DSF_ECUDA;
    }
    dz = laid_out(l->dtype, c.N) ? Mat{c.ws + c.w.gp, M, c.N, c.w.np, c.terms, M * c.w.np} : Mat{dy, M, c.N, lddy, 1, 0};
  }
  return grad_products(c, dz, dx, lddx, dW) ? DSF_OK : DSF_ECUDA;
}

int run_fwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const float* xs, const void* res,
            long long ldr, long long M, void* y, long long ldy, void* ws, size_t ws_bytes, int* status,
            void* stream) {
  if (int rc = check_layer(l, gated)) return rc;
  if (M < 0 || M > kMaxM) return DSF_EINVAL;
  if (M == 0) return DSF_OK;
  const int N = gated ? l->R / 2 : l->R, eo = osize(l->dtype);
  if (!rows_ok(x, ldx, l->K, esize(l->dtype))) return DSF_EINVAL;
  if ((l->dtype == DSF_E4M3) != (xs != nullptr) || !at(xs, 4)) return DSF_EINVAL;
  if (!y || ldy < N || !at(y, eo) || (res && (ldr < N || !at(res, eo)))) return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < ws_bytes_of(l, M, gated, false)) return DSF_EWORKSPACE;
  return fwd(l, gated, x, ldx, xs, res, ldr, M, y, ldy, ws, status, static_cast<cudaStream_t>(stream));
}

int run_bwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const void* dy, long long lddy, long long M,
            void* dx, long long lddx, void* dW, float* db, void* ws, size_t ws_bytes, int* status, void* stream) {
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
    if (dW && !succeeded(cudaMemsetAsync(dW, 0, size_t(l->R) * l->K * es, s))) return DSF_ECUDA;
    if (db && !succeeded(cudaMemsetAsync(db, 0, size_t(l->R) * 4, s))) return DSF_ECUDA;
    return DSF_OK;
  }
  return bwd(l, gated, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, status, s);
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
  return run_fwd(l, false, x, ldx, xs, res, ldr, M, y, ldy, ws, ws_bytes, status, stream);
}

int ctr_glu_fwd(const dsf_dense* l, const void* x, int64_t ldx, const float* xs, int64_t M, void* h, int64_t ldh,
                void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_fwd(l, true, x, ldx, xs, nullptr, 0, M, h, ldh, ws, ws_bytes, status, stream);
}

int ctr_dense_bwd(const dsf_dense* l, const void* x, int64_t ldx, const void* dy, int64_t lddy, int64_t M, void* dx,
                  int64_t lddx, void* dW, float* db, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_bwd(l, false, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, ws_bytes, status, stream);
}

int ctr_glu_bwd(const dsf_dense* l, const void* x, int64_t ldx, const void* dh, int64_t lddh, int64_t M, void* dx,
                int64_t lddx, void* dW, float* db, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_bwd(l, true, x, ldx, dh, lddh, M, dx, lddx, dW, db, ws, ws_bytes, status, stream);
}

}  // extern "C"
