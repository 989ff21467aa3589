// The softmax cross entropy of rows against a catalogue (ctr_softmax_xent_* in
// dinsparse.h): z = x W^T + bias over V columns, lse = log sum exp z, loss =
// lse - z_target, dz = g (exp(z - lse) - [v = target]), dx = dz W, dW = dz^T x,
// db = sum of dz.
//
// The logits are never kept. The forward is one pass of the product x W^T whose
// epilogue keeps a (reference, sum of exponentials) pair per row in registers over
// all of the tiles that a warp has of the row; a second kernel merges a row's pairs.
// Exponents are in units of log 2: exp(z - m) = 2^(z log2 e - m'), and m' is
// kept as it was subtracted, so its rounding cancels. The backward takes the
// catalogue in pieces: the product again, its epilogue writing the piece's dz
// (one rounding to bf16, or an fp32 operand's three terms), then dW's rows of
// the piece, complete, and dx added up over the pieces in fp32 planes. So
// memory holds M x (a piece), whatever V is, and sums run in a fixed order.
// (Pieces of 256 MB: 16384 rows, 65,536 columns of 1024 bf16, the sums and all
// gradients, 5.9 ms; of 64 MB 6.7, of 96 MB 6.5, of 1 GB 5.7.)
// Where x and W are narrow, passes that keep no dz at all take over (xent_pass.cuh),
// and few_kernel has the sums of a step of serving, 4 rows at most.
#include <climits>

#include "dense_host.cuh"
#include "xent_pass.cuh"

namespace dsf {
namespace dense {
namespace {

constexpr int kMaxK = 8192;
constexpr long long kMaxLogits = 1LL << 44;  // (2^30 tiles)
constexpr size_t kPieceBytes = 256u << 20;  // dz of a piece

// ---------------------------------------------------------------- small kernels
// A row's pairs [pairs][M] to lse and loss. `rows` (a power of two up to 32)
// neighbouring rows per block; the other threads share out the pairs.
constexpr int kWarpsPerRow = 4;
struct MergeArgs {
  const float2* stat;
  const float* zt;
  const long long* target;
  float *loss, *lse;
  long long M;
  int pairs, rows;
  long long V;
  int* status;
};
constexpr int kMerge = 256;
__global__ void __launch_bounds__(kMerge) merge_kernel(const __grid_constant__ MergeArgs a) {
  __shared__ float2 part[kMerge];
  pdl_go();
  pdl_wait();
  const int r = threadIdx.x & (a.rows - 1), slice = threadIdx.x / a.rows, slices = kMerge / a.rows;
  const long long row = (long long)blockIdx.x * a.rows + r;
  float m = -kFar, s = 0.f;
  if (row < a.M) {
    for (int k0 = slice; k0 < a.pairs; k0 += 4 * slices) {
      float2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * slices;
        p[u] = make_float2(-kFar, 0.f);
        if (k < a.pairs) p[u] = __ldg(a.stat + (long long)k * a.M + row);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float now = fmaxf(m, p[u].x);
        s = s * exp2_fast(m - now) + p[u].y * exp2_fast(p[u].x - now);
        m = now;
      }
    }
  }
  part[threadIdx.x] = make_float2(m, s);
  for (int n = slices / 2; n; n >>= 1) {
    __syncthreads();
    if (slice < n) {
      const float2 p = part[threadIdx.x], q = part[threadIdx.x + n * a.rows];
      const float now = fmaxf(p.x, q.x);
      part[threadIdx.x] = make_float2(now, p.y * exp2_fast(p.x - now) + q.y * exp2_fast(q.x - now));
    }
  }
  if (slice != 0 || row >= a.M) return;
  const float2 p = part[threadIdx.x];
  const float lse = (p.x + log2f(p.y)) * 0.69314718055994530942f;
  const long long t = a.target[row];
  const bool there = t >= 0 && t < a.V;
  a.lse[row] = lse;
  // (nothing possible: NaN, also where the target's logit is finite)
  a.loss[row] = !there ? 0.f : (lse == -INFINITY ? NAN : lse - a.zt[row]);
  if (!there && t != -1 && a.status) atomicOr(a.status, DSF_FLAG_ID_RANGE);
}

// The sums of up to MT rows from W's rows as they lie in memory, on the CUDA cores: a
// tensor-core tile would use MT of its 128 rows. The catalogue's bytes are what counts
// (one row, 846,812 x 64 bf16: 26 us with the merge; by tiles 44). 2^log_g lanes side
// by side have one row of W (a 16-byte vector each), a warp 32 / 2^log_g rows, and U
// of those in flight; each lane keeps the reference and sum of its rows (alike in the
// lanes of a row).
struct FewArgs {
  const void *x, *W;
  long long ldx, ldw;
  const float* bias;
  const long long* target;
  float2* stat;  // [blocks][M]
  float* zt;
  int M, V, nv, log_g;  // nv: vectors of a row
};
constexpr int kFewBlocks = 4 * kSms;
static_assert(kFewBlocks <= kLseClusters * kWarpsPerRow, "lse_room");
template <class T, int MT>
__global__ void __launch_bounds__(256) few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int E = 16 / int(sizeof(T)), U = 4;
  __shared__ float2 part[8][MT];
  pdl_go();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = 1 << a.log_g, at = lane & (g - 1);
  const bool live = at < a.nv;
  float x[MT][E];
  int tgt[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = min(m, a.M - 1);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (live) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + r * a.ldx) + at);
    unpack(v, x[m], T());
    const long long id = __ldg(a.target + r);
    tgt[m] = m < a.M && id >= 0 && id < a.V ? int(id) : -1;
  }
  float top[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) top[m] = -kFarthest, sum[m] = 0.f;
  const int per = 32 >> a.log_g;  // W's rows of a warp and step
  const long long step = (long long)gridDim.x * 8 * per;
  for (long long v0 = ((long long)blockIdx.x * 8 + warp) * per + (lane >> a.log_g); v0 - (lane >> a.log_g) < a.V; v0 += U * step) {
    uint4 w[U];
    float b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long v = v0 + u * step;
      w[u] = make_uint4(0, 0, 0, 0);
      if (live && v < a.V) w[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.W) + v * a.ldw) + at);
      b[u] = v < a.V ? (a.bias ? __ldg(a.bias + v) : 0.f) : -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long v = v0 + u * step;
      float wf[E];
      unpack(w[u], wf, T());
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(x[m][e], wf[e], z);
        for (int o = g / 2; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        z += b[u];
        if (v == tgt[m] && at == 0) a.zt[m] = z;
        const float zl = z * kLog2e, now = fmaxf(top[m], fminf(zl, kFarthest));
        sum[m] = sum[m] * exp2_fast(top[m] - now) + exp2_fast(zl - now);
        top[m] = now;
      }
    }
  }
  // over the warp's rows of W, the block's warps
  auto both = [](float2 p, float2 q) {
    const float now = fmaxf(p.x, q.x);
    return make_float2(now, p.y * exp2_fast(p.x - now) + q.y * exp2_fast(q.x - now));
  };
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float2 p = make_float2(top[m], sum[m]);
    for (int o = g; o < 32; o <<= 1)
      p = both(p, make_float2(__shfl_xor_sync(0xffffffffu, p.x, o), __shfl_xor_sync(0xffffffffu, p.y, o)));
    if (lane == 0) part[warp][m] = p;
  }
  __syncthreads();
  if (threadIdx.x < unsigned(a.M)) {
    float2 p = part[0][threadIdx.x];
    for (int k = 1; k < 8; ++k) p = both(p, part[k][threadIdx.x]);
    a.stat[(long long)blockIdx.x * a.M + threadIdx.x] = p;
  }
}

// What the backward's products take per row: lse in units of log 2 (kFar: the row is
// left out; also where no column is possible) and dloss; as pairs, or in one array
// each, with the target, up to a whole tile of 128 rows.
struct RowsArgs {
  const long long* target;
  const float *lse, *dloss;
  long long M, V;
  float2* rows;
  float *l, *g;
  int *id, *status;
};
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ RowsArgs a) {
  pdl_go();
  pdl_wait();
  const long long r = blockIdx.x * 256LL + threadIdx.x;
  bool there = false;
  float l = kFar, g = 0.f;
  long long t = -1;
  if (r < a.M) {
    t = a.target[r];
    l = a.lse[r];
    there = t >= 0 && t < a.V;
    if (!there && t != -1 && a.status) atomicOr(a.status, DSF_FLAG_ID_RANGE);
    if (l == -INFINITY) there = false;
    l = there ? l * kLog2e : kFar;
    g = there ? (a.dloss ? a.dloss[r] : 1.f) : 0.f;
    if (a.rows) a.rows[r] = make_float2(l, g);
  }
  if (a.l && r < (a.M + 127) / 128 * 128) {
    a.l[r] = l;
    a.g[r] = g;
    a.id[r] = there ? int(t) : -1;
  }
}

// A bias in whole tiles of 128
__global__ void __launch_bounds__(256) bias_kernel(const float* bias, int V, float* out) {
  pdl_go();
  pdl_wait();
  const int v = blockIdx.x * 256 + threadIdx.x;
  if (v < (V + 127) / 128 * 128) out[v] = v < V ? bias[v] : 0.f;
}

// db from its four parts
__global__ void __launch_bounds__(256) db_kernel(const float* part, int V, float* db) {
  pdl_go();
  pdl_wait();
  const int v = blockIdx.x * 256 + threadIdx.x;
  if (v < V) db[v] = (part[v] + part[V + v]) + (part[2LL * V + v] + part[3LL * V + v]);
}

// ---------------------------------------------------------------- layout
// Whether the rows' sums, or the gradients, are taken in one pass each (xent_pass.cuh):
// from 4e7 logits on, where the catalogue gives the SMs work (a unit of dW's pass is 128 of
// its rows); the sums of 1e8 in any case. (The gradients both ways, us, at K = 64: 512 rows
// over 100,000 columns 65 and 82, 2000 over 20,000 61 and 70, 64 over 846,812 172 and 199,
// 8192 over 8192 85 and 85, 20,000 over 6000 182 and 155; at K = 128: 128 rows over
// 1,000,000 295 and 320, 512 over 100,000 81 and 94. The sums of those: 44 and 49, 42 and
// 46, 68 and 72, 53 and 61, 77 and 92; 81 and 82, 46 and 48.)
bool narrow(const dsf_dense* l, long long M, bool backward) {
  const double logits = double(M) * l->R;
  return l->dtype == DSF_BF16 && l->K <= 128 && M <= 65536 && ((logits >= 1e8 && !backward) || (l->R >= 8192 && logits >= 4e7));
}
// Whether the sums are few_kernel's: of up to 4 rows, whole vectors, at most 32 of them.
bool few(const dsf_dense* l, long long M) {
  const int bytes = l->K * esize(l->dtype);
  return M <= 4 && bytes % 16 == 0 && bytes <= 512;
}
// Chunks of the columns in which the sums and dx are taken: at most 512 tiles in one, and
// units whose whole rounds over the SMs take the least time (a unit costs 6 tiles more).
constexpr int kDxRounds = 8;
constexpr long long kDxUnits = kDxRounds * kSms;
int dx_chunks(long long M, long long V) {
  const long long mt = (M + 127) / 128, ct = (V + 127) / 128, least = (ct + 511) / 512;
  long long best = least, time = LLONG_MAX;
  for (int r = 0; r <= kDxRounds; ++r) {  // (the most chunks in r rounds; the fewest there can be)
    const long long most = r * kSms / mt, c = r == 0 || most < least ? least : (most < ct ? most : ct);
    const long long per = (ct + c - 1) / c, units = mt * ((ct + per - 1) / per), t = (units + kSms - 1) / kSms * (per + 6);
    if (t < time) best = c, time = t;
  }
  return int(best);
}

// Columns of a piece for M rows.
long long piece_of(const dsf_dense* l, long long M) {
  const long long terms = l->dtype == DSF_F32 ? 3 : 1, all = up(l->R, 256);
  const long long p = (long long)(kPieceBytes / (2 * size_t(terms) * size_t(M))) / 256 * 256;
  return p < 256 ? 256 : (p < all ? p : all);
}

struct XLayout {
  size_t xp, wp, bias, stat, zt, rows, dz, sums, part, planes, total;
  long long kp;
};
XLayout xent_layout(const dsf_dense* l, long long M, bool backward) {
  XLayout w{};
  const bool f32 = l->dtype == DSF_F32;
  const size_t terms = f32 ? 3 : 1, m = size_t(M);
  w.kp = up(l->K, 8);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t here = o;
    o += align256(bytes);
    return here;
  };
  const bool lo = laid_out(l->dtype, l->K);
  w.xp = take(lo || backward ? terms * m * w.kp * 2 : 0);
  w.wp = take(lo ? terms * size_t(l->R) * w.kp * 2 : 0);
  size_t stat = size_t(lse_room(M)) * kWarpsPerRow * 8;  // (few_kernel's blocks: as many pairs of up to 4 rows)
  const bool by_pass = l->dtype == DSF_BF16 && l->K <= 128;  // (for some number of rows)
  const size_t mt = (m + 127) / 128, pieces = 128 * (size_t(kDxUnits) + mt);  // rows times chunks, at most these or 16 times the rows
  if (by_pass && stat < (pieces > m * 16 ? pieces : m * 16) * kWarpsPerRow * 8)
    stat = (pieces > m * 16 ? pieces : m * 16) * kWarpsPerRow * 8;
  w.bias = take(by_pass && l->bias ? size_t(up(l->R, 128)) * 4 : 0);
  // the forward's and the backward's scratch share their room
  size_t o0 = o;
  w.stat = take(stat);
  w.zt = take(m * 4);
  size_t most = o;
  if (backward) {
    o = o0;
    const size_t all = size_t(up(l->R, 256)), K4 = size_t(up(l->K, 4)) * 4;
    auto least = [](size_t a, size_t b) { return a < b ? a : b; };
    auto greatest = [](size_t a, size_t b) { return a > b ? a : b; };
    // (each is at least what any smaller M takes: a piece is at most kPieceBytes of dz, or 256 columns)
    w.rows = take((m + 128) * 12);
    w.dz = take(least(2 * terms * m * all, greatest(kPieceBytes, 2 * terms * m * 256)));
    w.sums = take(greatest(all * 16, least((m + 31) / 32 * all * 4, kPieceBytes / 16 / terms + (m + 31) / 32 * 256 * 4 + all * 4)));
    // planes of dx: the splits of a product, or those of sums of more than 65536 terms
    const size_t outputs = m * K4;
    const size_t planes = greatest(least(outputs * kMaxSplits, kPartBytes), outputs + K4 * (kPieceBytes / 131072 + 1));
    w.planes = take(by_pass ? greatest(planes, greatest(pieces * K4, outputs * 16)) : planes);  // (dx_chunks of them)
    // partial sums of dW's rows of a piece, or, where one piece is all, of dx
    const size_t wide = all * K4;
    w.part = take(greatest(greatest(least(wide * kMaxSplits, kPartBytes), planes),
                           M > 65536 ? least(wide, K4 * (256 + kPieceBytes / 2 / 65536)) * kMaxSplits : 0));
    most = most > o ? most : o;
  }
  w.total = most + 256;
  return w;
}

// ---------------------------------------------------------------- products
// The logits' tiles: 256 or 128 rows. (The narrow one where few rows leave
// half of the wide one empty.)
void plan_xent(Product& p, long long M, long long N, long long nkb) {
  const Cost cost{p.f32};
  double best = 1e300;
  Job o = p.a.job[0];
  for (int cfg = 0; cfg < 2; ++cfg) {
    set_tiles(o, cfg, M, N, 1, false, p.f32, nkb, 1, 1);
    const long long waves = (tiles_of(o) + slots_of(cfg) - 1) / slots_of(cfg);
    const double c = cost.run(cfg, double(waves), double(o.kbps));
    if (c < best) {
      best = c;
      p.cfg = cfg;
      p.a.job[0] = o;
    }
  }
}

// Whether dx and dW are best made in one launch, where dx's sums (over the
// columns) are not split: with few rows and many columns each of its few tiles
// would take all of them in turn (500 x 176 fp32 over 12,961 columns: 200 us in
// one launch).
bool together(long long M, long long N, long long K, bool f32) {
  Product p{}, q{}, r{};
  p.f32 = q.f32 = r.f32 = f32;
  p.epi = q.epi = r.epi = kEpiOut;
  return plan_dual(p, M, N, K, 1) <= plan(q, N, K, 1, (M + 63) / 64, 1, true) + plan(r, M, K, 1, (N + 63) / 64, 1, true);
}

bool merge(MergeArgs g, cudaStream_t s) {
  while (g.rows > 1 && g.rows / 2 >= g.M) g.rows /= 2;
  while (g.rows > 4 && (g.M + g.rows - 1) / g.rows < 2 * kSms) g.rows /= 2;
  return pdl_launch(merge_kernel, dim3(unsigned((g.M + g.rows - 1) / g.rows)), kMerge, s, g);
}

// The bias as the passes take it, where there is one
bool lay_bias(const dsf_dense* l, void* ws, const float** bias, cudaStream_t s) {
  *bias = l->bias ? static_cast<const float*>(ws) : nullptr;
  return !l->bias || pdl_launch(bias_kernel, dim3(unsigned((l->R + 127 + 255) / 256)), 256, s, l->bias, l->R, static_cast<float*>(ws));
}

bool xent_fwd(const dsf_dense* l, const void* x, long long ldx, const long long* target, long long M, float* loss,
              float* lse, uint8_t* ws, int* status, cudaStream_t s) {
  const bool f32 = l->dtype == DSF_F32, lo = laid_out(l->dtype, l->K);
  const XLayout w = xent_layout(l, M, false);
  const int terms = f32 ? 3 : 1;
  if (lo && !few(l, M)) {
    const LayJob jobs[2] = {{x, ws + w.xp, ldx, M, w.kp, l->K, nullptr, 0},
                            {l->W, ws + w.wp, l->ldw, l->R, w.kp, l->K, nullptr, 0}};
    if (!lay(l->dtype, jobs, 2, s)) return false;
  }
  float2* stat = reinterpret_cast<float2*>(ws + w.stat);
  float* zt = reinterpret_cast<float*>(ws + w.zt);
  if (few(l, M)) {
    FewArgs a{x, l->W, ldx, l->ldw, l->bias, target, stat, zt, int(M), l->R, l->K * esize(l->dtype) / 16, 0};
    while ((1 << a.log_g) < a.nv) ++a.log_g;
    const long long steps = ((long long)l->R * (1 << a.log_g) + 255) / 256;  // (a block's rows of W in a step)
    const int blocks = int(steps < kFewBlocks ? steps : kFewBlocks);
    const bool ok = f32 ? (M == 1 ? pdl_launch(few_kernel<float, 1>, dim3(unsigned(blocks)), 256, s, a)
                                  : pdl_launch(few_kernel<float, 4>, dim3(unsigned(blocks)), 256, s, a))
                        : (M == 1 ? pdl_launch(few_kernel<__nv_bfloat16, 1>, dim3(unsigned(blocks)), 256, s, a)
                                  : pdl_launch(few_kernel<__nv_bfloat16, 4>, dim3(unsigned(blocks)), 256, s, a));
    return ok && merge(MergeArgs{stat, zt, target, loss, lse, M, blocks, 32, l->R, status}, s);
  }
  if (narrow(l, M, false)) {
    PassArgs a{};
    const float* bias = nullptr;
    if (!lay_bias(l, ws + w.bias, &bias, s)) return false;
    a.R = int(M), a.C = l->R, a.K = l->K;
    a.rt = int((M + 127) / 128), a.ct = int((l->R + 127) / 128);
    const int chunks = dx_chunks(M, l->R);
    a.per = (a.ct + chunks - 1) / chunks;
    a.chunks = (a.ct + a.per - 1) / a.per;
    a.col0 = bias;
    a.target = target;
    a.stat = stat;
    a.zt = zt;
    a.status = status;
    const Mat X = lo ? Mat{ws + w.xp, M, l->K, w.kp, 1, 0} : Mat{x, M, l->K, ldx, 1, 0},
              W = lo ? Mat{ws + w.wp, l->R, l->K, w.kp, 1, 0} : Mat{l->W, l->R, l->K, l->ldw, 1, 0};
    return run_xent_pass(kSums, a, X, W, s) &&
           merge(MergeArgs{stat, zt, target, loss, lse, M, kWarpsPerRow * a.chunks, 32, l->R, status}, s);
  }
  Product p{};
  p.A = lo ? Mat{ws + w.xp, M, l->K, w.kp, terms, M * w.kp} : Mat{x, M, l->K, ldx, 1, 0};
  p.B = lo ? Mat{ws + w.wp, l->R, l->K, w.kp, terms, l->R * w.kp} : Mat{l->W, l->R, l->K, l->ldw, 1, 0};
  p.major = kKK;
  p.f32 = f32;
  p.epi = kEpiLse;
  p.a.job[0].a_term = p.a.job[0].b_term = 1;
  plan_xent(p, M, l->R, (l->K + 63) / 64);
  p.a.bias = l->bias;
  p.a.target = target;
  p.a.stat = stat;
  p.a.zt = zt;
  p.a.status = status;
  int slots = 0;
  p.lse_slots = &slots;
  if (!run_xent_product(p, s)) return false;
  return merge(MergeArgs{stat, zt, target, loss, lse, M, kWarpsPerRow * slots, 32, l->R, status}, s);
}

bool xent_bwd(const dsf_dense* l, const void* x, long long ldx, const long long* target, const float* lse,
              const float* dloss, long long M, void* dx, long long lddx, void* dW, float* db, uint8_t* ws, int* status,
              cudaStream_t s) {
  const bool f32 = l->dtype == DSF_F32, lo = laid_out(l->dtype, l->K);
  const XLayout w = xent_layout(l, M, true);
  const int terms = f32 ? 3 : 1, es = esize(l->dtype), K = l->K;
  // x with the rows that are left out as zeros: their dz is zero, and dW adds
  // dz x, whatever x holds there
  const LayJob jobs[2] = {{x, ws + w.xp, ldx, M, w.kp, K, target, l->R},
                          {l->W, ws + w.wp, l->ldw, l->R, w.kp, K, nullptr, 0}};
  if (!lay(l->dtype, jobs, lo ? 2 : 1, s)) return false;
  const bool pass = narrow(l, M, true);
  const long long Mp = up(M, 128);
  float* l_of = reinterpret_cast<float*>(ws + w.rows);
  float2* rows = pass ? nullptr : reinterpret_cast<float2*>(l_of);
  RowsArgs ra{target, lse, dloss, M, l->R, rows, pass ? l_of : nullptr, l_of + Mp, reinterpret_cast<int*>(l_of + 2 * Mp), status};
  if (!pdl_launch(rows_kernel, dim3(unsigned((Mp + 255) / 256)), 256, s, ra)) return false;
  float* sums = reinterpret_cast<float*>(ws + w.sums);
  Ctx c{};
  c.l = l;
  c.M = M;
  c.halves = 1;
  c.es = c.eo = es;
  c.terms = terms;
  c.kbe = 64;
  c.ws = ws;
  c.w.part = w.part;
  c.status = status;
  c.s = s;
  c.X = Mat{ws + w.xp, M, K, w.kp, terms, M * w.kp};
  if (pass) {
    c.W = lo ? Mat{ws + w.wp, l->R, K, w.kp, 1, 0} : Mat{l->W, l->R, K, l->ldw, 1, 0};
    const int mt = int(Mp / 128), vt = int((l->R + 127) / 128);
    if (dW || db) {
      PassArgs g{};
      g.K = K, g.status = status;
      g.R = l->R, g.C = int(M), g.rt = vt, g.ct = mt;
      g.chunks = 1, g.per = mt;
      g.col0 = ra.l, g.col1 = ra.g, g.col_id = ra.id;
      g.row0 = l->bias;
      g.out = dW, g.ldo = K;
      g.db = db ? sums : nullptr;
      if (!run_xent_pass(kDw, g, c.W, c.X, s)) return false;
      if (db && !pdl_launch(db_kernel, dim3(unsigned((l->R + 255) / 256)), 256, s, (const float*)sums, l->R, db)) return false;
    }
    if (!dx) return true;
    PassArgs g{};
    const float* bias = nullptr;
    if (!lay_bias(l, ws + w.bias, &bias, s)) return false;
    const int chunks = dx_chunks(M, l->R);
    g.K = K, g.status = status;
    g.R = int(M), g.C = l->R, g.rt = mt, g.ct = vt;
    g.per = (vt + chunks - 1) / chunks;
    g.chunks = (vt + g.per - 1) / g.per;
    g.col0 = bias;
    g.row0 = ra.l, g.row1 = ra.g, g.target = target;
    g.out = ws + w.planes;
    g.ldo = up(K, 4);
    g.plane = M * g.ldo;
    if (!run_xent_pass(kDx, g, c.X, c.W, s)) return false;
    Product sum{};
    Job& o = sum.a.job[0];
    o.M = int(M), o.N = K, o.splits = g.chunks, o.ldo = g.ldo;
    c.w.part = w.planes;
    FinishArgs f{};
    f.planes = 1;
    f.out = dx;
    f.ldo = lddx;
    return finish(c, sum, f, false);
  }
  const long long P = piece_of(l, M);
  const bool one = P >= l->R;
  Product acc{};  // dx over the pieces: the first piece's plan for all of them
  int planes = 0;
  for (long long v = 0; v < l->R; v += P) {
    const long long n = l->R - v < P ? l->R - v : P, np = up(n, 8);
    c.N = int(n);
    c.W = lo ? Mat{ws + w.wp + v * w.kp * 2, n, K, w.kp, terms, l->R * w.kp}
             : Mat{static_cast<const uint8_t*>(l->W) + v * l->ldw * es, n, K, l->ldw, 1, 0};
    const Mat dz{ws + w.dz, M, n, np, terms, M * np};
    Product p{};
    p.A = c.X;
    p.B = c.W;
    p.major = kKK;
    p.f32 = f32;
    p.epi = kEpiXent;
    p.a.job[0].a_term = p.a.job[0].b_term = 1;
    plan_xent(p, M, n, (K + 63) / 64);
    p.a.bias = l->bias ? l->bias + v : nullptr;
    p.a.part = db ? sums : nullptr;
    p.a.target = target;
    p.a.v0 = int(v);
    p.a.rows = rows;
    p.a.status = status;
    set_out(p.a.job[0], ws + w.dz, np, 2);
    if (!run_xent_product(p, s)) return false;
    if (db && !colsum(sums, (M + 31) / 32, int(n), db + v, s)) return false;
    void* dWv = dW ? static_cast<uint8_t*>(dW) + v * K * es : nullptr;
    // (apart, too, where larger calls take a pass each: no output then depends on which are asked for)
    if (one && dx && dWv && (narrow(l, M, false) || !together(M, n, K, f32))) {
      if (!grad_products(c, dz, nullptr, 0, dWv)) return false;
      return grad_products(c, dz, dx, lddx, nullptr);
    }
    if (one) return grad_products(c, dz, dx, lddx, dWv);
    if (dWv && !grad_products(c, dz, nullptr, 0, dWv)) return false;
    if (!dx) continue;
    const long long nkb = (n + 63) / 64;
    Job& o = acc.a.job[0];
    if (v == 0) {
      acc.major = kKN;
      acc.f32 = f32;
      acc.a.status = status;
      plan(acc, M, K, 1, nkb, 1, true);
      planes = o.splits;
      acc.epi = kEpiPart;
    } else {
      acc.epi = kEpiAcc;
      set_tiles(o, acc.cfg, M, K, 1, false, f32, nkb, 1, planes);
    }
    o.a_term = o.b_term = o.a_seg = 1;
    o.out = ws + w.planes;
    o.ldo = up(K, 4);
    o.out_plane = M * o.ldo;
    o.out_vec = 1;
    acc.A = dz;
    acc.B = c.W;
    acc.a.in = o.out;
    acc.a.ldi = o.ldo;
    acc.a.in_vec = 1;
    if (!(v == 0 ? run_grad_product(acc, s) : run_acc_product(acc, s))) return false;
  }
  if (!dx) return true;
  c.w.part = w.planes;
  acc.a.job[0].splits = planes;
  FinishArgs f{};
  f.planes = 1;
  f.out = dx;
  f.ldo = lddx;
  return finish(c, acc, f, f32);
}

// ---------------------------------------------------------------- checks
int check_xent(const dsf_dense* l) {
  if (int rc = check_layer(l, false)) return rc;
  if (l->dtype == DSF_E4M3 || l->K > kMaxK) return DSF_EUNSUPPORTED;
  return l->act == DSF_ACT_NONE ? DSF_OK : DSF_EINVAL;
}
int check_rows(const dsf_dense* l, int64_t M) {
  if (M < 0 || M > kMaxM) return DSF_EINVAL;
  return M > kMaxLogits / l->R ? DSF_EUNSUPPORTED : DSF_OK;
}

}  // namespace
}  // namespace dense
}  // namespace dsf

using namespace dsf::dense;

extern "C" {

size_t dsf_softmax_xent_workspace_bytes(const dsf_dense* l, int64_t M, int32_t backward) {
  if (check_xent(l) != DSF_OK || check_rows(l, M) != DSF_OK || backward < 0 || backward > 1) return 0;
  return xent_layout(l, M, backward != 0).total;
}

int ctr_softmax_xent_fwd(const dsf_dense* l, const void* x, int64_t ldx, const int64_t* target, int64_t M, float* loss,
                         float* lse, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  if (int rc = check_xent(l)) return rc;
  if (int rc = check_rows(l, M)) return rc;
  if (M == 0) return DSF_OK;
  if (!rows_ok(x, ldx, l->K, esize(l->dtype)) || !target || !at(target, 8) || !loss || !at(loss, 4) || !lse || !at(lse, 4))
    return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < xent_layout(l, M, false).total) return DSF_EWORKSPACE;
  return xent_fwd(l, x, ldx, reinterpret_cast<const long long*>(target), M, loss, lse, static_cast<uint8_t*>(ws), status,
                  static_cast<cudaStream_t>(stream))
             ? DSF_OK
             : DSF_ECUDA;
}

int ctr_softmax_xent_bwd(const dsf_dense* l, const void* x, int64_t ldx, const int64_t* target, const float* lse,
                         const float* dloss, int64_t M, void* dx, int64_t lddx, void* dW, float* db, void* ws,
                         size_t ws_bytes, int32_t* status, void* stream) {
  if (int rc = check_xent(l)) return rc;
  if (int rc = check_rows(l, M)) return rc;
  const int es = esize(l->dtype);
  if (!at(dW, es) || !at(db, 4)) return DSF_EINVAL;
  if (M > 0 && (!rows_ok(x, ldx, l->K, es) || !target || !at(target, 8) || !lse || !at(lse, 4) || !at(dloss, 4) ||
                (dx && (lddx < l->K || !at(dx, es)))))
    return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < xent_layout(l, M, true).total) return DSF_EWORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dW && !dsf::succeeded(cudaMemsetAsync(dW, 0, size_t(l->R) * l->K * es, s))) return DSF_ECUDA;
    if (db && !dsf::succeeded(cudaMemsetAsync(db, 0, size_t(l->R) * 4, s))) return DSF_ECUDA;
    return DSF_OK;
  }
  if (!dx && !dW && !db) return DSF_OK;
  return xent_bwd(l, x, ldx, reinterpret_cast<const long long*>(target), lse, dloss, M, dx, lddx, dW, db,
                  static_cast<uint8_t*>(ws), status, s)
             ? DSF_OK
             : DSF_ECUDA;
}

}  // extern "C"
