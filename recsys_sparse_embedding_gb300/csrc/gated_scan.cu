// The gated linear recurrence over jagged sequences and its gradients
// (ctr_gated_scan_* in dinsparse.h).
//
//   forward   h_t = a_t h_{t-1} + z_t x_t,      z = sigmoid(gate), a = 1 - z
//   backward  g_t = dh_t + c_{t+1},  c_t = a_t g_t;  dx = g z,
//             dgate = g (x - h_{t-1}) z a,      dh0 = c at a sequence's first row
//
// Both are first-order recurrences y_t = A_t y_{t-1} + B_t (the backward with
// rows in descending order: c_t = a_t c_{t+1} + a_t dh_t), and pairs (A, B)
// compose. Rows are taken as one stream in which a sequence's first row is a
// reset (its state comes from h0), so jagged lengths cost nothing.
//
// One pass over memory: a block holds a chunk of rows by up to 64 channels in
// registers (256 threads: V channels by NT rows each; the threads' row ranges
// are composed by shuffles and shared memory), publishes the chunk's pair,
// takes the pairs of the chunks before it as far as its first sequence
// reaches, and then writes its rows. Without the chain (a pass for the pairs,
// a second over x and gate) a long sequence would move 5/3 of the bytes.
// Fixed order: chunks are in groups of 32; a chunk starts from the state at
// the end of the group before its own and composes the pairs of its group in
// a fixed tree, so equal calls give equal bits, however blocks are scheduled,
// and the chain through memory has one step per group. Blocks take their
// chunks by a ticket, so a block only waits for blocks that have started;
// every wait is bounded and sets DSF_FLAG_TIMEOUT when it runs out.
//
// A reset is carried as A = -1 (A is never negative otherwise): nothing is
// multiplied across a sequence's border, so a non-finite state stays in its
// own sequence. States, pairs and sums are fp32; h, dx and dgate are rounded
// once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dinsparse.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace dsf {
namespace scan {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroup = 32;          // chunks per group
constexpr int kFwdRows = 8, kBwdRows = 4;  // rows per thread
constexpr int kMaxDim = 1 << 20;
constexpr long long kMaxRows = 1 << 30;

struct Args {
  const void *x, *gate, *h, *dh;  // h, dh: backward
  void *o0, *o1;                  // h; dx and dgate
  long long ldx, ldg, ldh, lddh, ldo0, ldo1;
  const float* in;  // [B, D]: h0; dh_last (nullable)
  const float* h0;  // backward: [B, D] (nullable)
  float* out;       // [B, D]: h_last; dh0 (nullable)
  const int* off;   // [B + 1] first rows of the sequences; null: equal lengths L
  const int* first; // [chunks + 1]: the sequence of a chunk's first row
  int T, B, D, L;
  int chunks, tiles, log_ct;
  int chain;  // whether a sequence may go on from chunk to chunk
  uint32_t *ticket, *flags, *group_flags;  // flags: [chunks][tiles]; group_flags: [groups][tiles]
  float2* pairs;                           // [chunks][tiles][CT V]
  float* states;                           // [groups][tiles][CT V]
  int* status;
};

// V neighbouring elements of a row
template <class T, int V>
struct Raw;
template <>
struct Raw<float, 4> {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ void get(float* f) const { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }
  static __device__ void put(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 v = make_uint2(0, 0);
  __device__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ void get(float* f) const {
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  static __device__ void put(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
};
template <class T>
struct Raw<T, 1> {
  T v = T(0.f);
  __device__ void load(const T* p) { v = *p; }
  __device__ void get(float* f) const { f[0] = float(v); }
  static __device__ void put(T* p, const float* f) { *p = T(f[0]); }
};

// z = sigmoid(g) and a = 1 - z, both to a few last bits of their own size
__device__ __forceinline__ void gate_of(float g, float& z, float& a) {
  const float t = __expf(-fabsf(g)), r = __fdividef(1.f, 1.f + t), s = t * r;
  z = g >= 0.f ? r : s;
  a = g >= 0.f ? s : r;
  if (g != g) z = a = g;
}

// (A, B) := (A, B) after (Ap, Bp)
__device__ __forceinline__ void compose(float Ap, float Bp, float& A, float& B) {
  if (A < 0.f) return;
  B = fmaf(A, Bp, B);
  A = Ap < 0.f ? -1.f : A * Ap;
}
__device__ __forceinline__ float apply(float A, float B, float y) { return A < 0.f ? B : fmaf(A, y, B); }

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Waits until *p is set; false after about a second.
__device__ bool wait_set(const uint32_t* p) {
  if (ld_acquire(p)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!ld_acquire(p))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

template <class T, int V, int NT, bool REV>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(const __grid_constant__ Args a) {
  constexpr int kMaxC = kThreads / 4 * NT;
  __shared__ int s_start[kMaxC], s_end[kMaxC];  // the sequence that a row is the first (last) of, or -1
  __shared__ float2 s_pair[kWarps][64], s_look[kWarps][64];
  __shared__ float s_carry[64];
  __shared__ int s_idx;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int CT = 1 << a.log_ct, ct = tid & (CT - 1), slice = tid >> a.log_ct, TS = kThreads >> a.log_ct, C = TS * NT;
  pdl_go();
  pdl_wait();
  int idx = blockIdx.x;
  if (a.chain) {
    if (tid == 0) s_idx = int(atomicAdd(a.ticket, 1u));
    __syncthreads();
    idx = s_idx;
  }
  const int rank = idx / a.tiles, tile = idx - rank * a.tiles, chunk = REV ? a.chunks - 1 - rank : rank;
  const int total = a.off ? a.off[a.B] : a.T, t0 = chunk * C;
  if (t0 >= total) return;
  const int n = min(C, total - t0), c0 = (tile * CT + ct) * V;
  const bool live = c0 < a.D;
  // the thread's rows, in scan order: row u0 + i of the chunk, or from its end
  auto row_of = [&](int i) { return REV ? C - 1 - (slice * NT + i) : slice * NT + i; };

  Raw<T, V> rx[NT], rg[NT], rh[REV ? NT : 1], rd[REV ? NT : 1];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int k = row_of(i);
    if (!live || k >= n) continue;
    const long long t = t0 + k;
    rx[i].load(static_cast<const T*>(a.x) + t * a.ldx + c0);
    rg[i].load(static_cast<const T*>(a.gate) + t * a.ldg + c0);
    if (REV) {
      rd[REV ? i : 0].load(static_cast<const T*>(a.dh) + t * a.lddh + c0);
      if (t > 0) rh[REV ? i : 0].load(static_cast<const T*>(a.h) + (t - 1) * a.ldh + c0);
    }
  }
  // where sequences start and end
  int from = 0;  // ragged: the sequence of the chunk's first row
  if (a.off) {
    from = a.first[chunk];
    for (int k = tid; k < C; k += kThreads) s_start[k] = s_end[k] = -1;
    __syncthreads();
    for (int s = from + tid; s < a.B; s += kThreads) {
      const int b = a.off[s], e = a.off[s + 1];
      if (b >= t0 + n) break;
      if (e == b) continue;
      if (b >= t0) s_start[b - t0] = s;
      if (e <= t0 + n) s_end[e - 1 - t0] = s;
    }
  } else {
    for (int k = tid; k < C; k += kThreads) {
      const int t = t0 + k, s = t / a.L, r = t - s * a.L;
      s_start[k] = r == 0 ? s : -1;
      s_end[k] = r == a.L - 1 ? s : -1;
    }
  }
  __syncthreads();

  // the rows' pairs, and what the outputs take besides
  float A[NT][V], Bv[NT][V], w[REV ? NT : 1][V], z[REV ? NT : 1][V];  // REV: Bv is dh
  uint32_t reset = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int k = row_of(i);
    const bool in = live && k < n;
    float x[V], g[V];
    rx[i].get(x);
    rg[i].get(g);
    const int seq = in ? (REV ? s_end[k] : s_start[k]) : -1;
    if (seq >= 0) reset |= 1u << i;
    float s[V], hp[V], d[V];
    Raw<float, V> state;
    if (seq >= 0 && a.in) state.load(a.in + (long long)seq * a.D + c0);
    state.get(s);
    if (REV) {
      rh[REV ? i : 0].get(hp);
      rd[REV ? i : 0].get(d);
      const int b = in ? s_start[k] : -1;
      if (b >= 0) {
        Raw<float, V> r;
        if (a.h0) r.load(a.h0 + (long long)b * a.D + c0);
        r.get(hp);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float zz, aa;
      gate_of(g[v], zz, aa);
      if (REV) {
        A[i][v] = in ? aa : 1.f;
        Bv[i][v] = in ? d[v] + s[v] : 0.f;
        w[REV ? i : 0][v] = (x[v] - hp[v]) * (zz * aa);
        z[REV ? i : 0][v] = zz;
      } else {
        A[i][v] = in ? aa : 1.f;
        Bv[i][v] = in ? (seq >= 0 ? fmaf(aa, s[v], zz * x[v]) : zz * x[v]) : 0.f;
      }
    }
  }
  // the thread's pair, then the pairs of the threads before it
  float PA[V], PB[V];
#pragma unroll
  for (int v = 0; v < V; ++v) PA[v] = 1.f, PB[v] = 0.f;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool r = reset >> i & 1;
      if (REV) PB[v] = A[i][v] * (r ? Bv[i][v] : PB[v] + Bv[i][v]);
      else PB[v] = r ? Bv[i][v] : fmaf(A[i][v], PB[v], Bv[i][v]);
      PA[v] = r || PA[v] < 0.f ? -1.f : PA[v] * A[i][v];
    }
  auto warp_scan = [&](float* qa, float* qb) {  // inclusive, over the warp's slices
    for (int d = CT; d < 32; d <<= 1)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float ap = __shfl_up_sync(0xffffffffu, qa[v], d), bp = __shfl_up_sync(0xffffffffu, qb[v], d);
        if (lane >= d) compose(ap, bp, qa[v], qb[v]);
      }
  };
  warp_scan(PA, PB);
  if (lane >= 32 - CT)
#pragma unroll
    for (int v = 0; v < V; ++v) s_pair[warp][ct * V + v] = make_float2(PA[v], PB[v]);
  // exclusive within the warp
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float ap = __shfl_up_sync(0xffffffffu, PA[v], CT & 31), bp = __shfl_up_sync(0xffffffffu, PB[v], CT & 31);
    PA[v] = lane >= CT ? ap : 1.f;
    PB[v] = lane >= CT ? bp : 0.f;
  }
  __syncthreads();
  float WA[V], WB[V], SA[V], SB[V];  // the pairs of the warps before this one; of the block
#pragma unroll
  for (int v = 0; v < V; ++v) {
    SA[v] = 1.f, SB[v] = 0.f, WA[v] = 1.f, WB[v] = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k == warp) WA[v] = SA[v], WB[v] = SB[v];
      float2 p = s_pair[k][ct * V + v];
      compose(SA[v], SB[v], p.x, p.y);
      SA[v] = p.x, SB[v] = p.y;
    }
    compose(WA[v], WB[v], PA[v], PB[v]);
  }

  // the chain: what goes on to the next chunk, and what comes from the last
  const bool goes_on = a.chain && (REV ? t0 > 0 && s_start[0] < 0 : t0 + n < total && s_end[n - 1] < 0);
  const bool comes_in = a.chain && (REV ? s_end[n - 1] < 0 : s_start[0] < 0);
  const int W = CT * V, group = rank / kGroup;
  bool ok = true;
  if (goes_on && warp == 0) {
    if (lane < CT && live)
#pragma unroll
      for (int v = 0; v < V; ++v)
        __stcg(&a.pairs[((long long)rank * a.tiles + tile) * W + ct * V + v], make_float2(SA[v], SB[v]));
    __threadfence();
    __syncwarp();
    if (lane == 0) st_release(a.flags + (long long)rank * a.tiles + tile, 1u);
  }
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.f;
  if (comes_in) {
    // the chunk where the chunk's first sequence (in scan order) begins
    int begin;
    if (a.off) {
      const int s = REV ? a.first[chunk + 1] : from;
      begin = REV ? a.chunks - 1 - (a.off[s + 1] - 1) / C : a.off[s] / C;
    } else {
      const int s = (REV ? t0 + n - 1 : t0) / a.L;
      begin = REV ? a.chunks - 1 - (s * a.L + a.L - 1) / C : s * a.L / C;
    }
    const int lo = max(begin, group * kGroup), count = rank - lo;
    const int each = (kGroup + TS - 1) / TS;
    float QA[V], QB[V];
#pragma unroll
    for (int v = 0; v < V; ++v) QA[v] = 1.f, QB[v] = 0.f;
    for (int j = slice * each; j < min(count, (slice + 1) * each); ++j) {
      const long long at = (long long)(lo + j) * a.tiles + tile;
      ok = wait_set(a.flags + at) && ok;
      if (live)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float2 p = __ldcg(&a.pairs[at * W + ct * V + v]);
          compose(QA[v], QB[v], p.x, p.y);
          QA[v] = p.x, QB[v] = p.y;
        }
    }
    __syncwarp();
    warp_scan(QA, QB);
    if (lane >= 32 - CT)
#pragma unroll
      for (int v = 0; v < V; ++v) s_look[warp][ct * V + v] = make_float2(QA[v], QB[v]);
    __syncthreads();
    if (tid < CT) {
      const long long at = (long long)(group - 1) * a.tiles + tile;
      const bool before = begin < group * kGroup;
      if (before) ok = wait_set(a.group_flags + at) && ok;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float y = before && live ? __ldcg(&a.states[at * W + ct * V + v]) : 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float2 p = s_look[k][ct * V + v];
          y = apply(p.x, p.y, y);
        }
        s_carry[ct * V + v] = y;
      }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = s_carry[ct * V + v];
  }
  if (goes_on && rank % kGroup == kGroup - 1 && warp == 0) {
    if (lane < CT && live)
#pragma unroll
      for (int v = 0; v < V; ++v)
        __stcg(&a.states[((long long)group * a.tiles + tile) * W + ct * V + v], apply(SA[v], SB[v], carry[v]));
    __threadfence();
    __syncwarp();
    if (lane == 0) st_release(a.group_flags + (long long)group * a.tiles + tile, 1u);
  }
  if (!ok && a.status) atomicOr(a.status, DSF_FLAG_TIMEOUT);
  if (!live) return;

  float y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) y[v] = apply(PA[v], PB[v], carry[v]);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int k = row_of(i);
    if (k >= n) continue;
    const long long t = t0 + k;
    const bool r = reset >> i & 1;
    if (REV) {
      float dx[V], dg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = r ? Bv[i][v] : Bv[i][v] + y[v];
        dx[v] = g * z[REV ? i : 0][v];
        dg[v] = g * w[REV ? i : 0][v];
        y[v] = A[i][v] * g;
      }
      Raw<T, V>::put(static_cast<T*>(a.o0) + t * a.ldo0 + c0, dx);
      Raw<T, V>::put(static_cast<T*>(a.o1) + t * a.ldo1 + c0, dg);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = r ? Bv[i][v] : fmaf(A[i][v], y[v], Bv[i][v]);
      Raw<T, V>::put(static_cast<T*>(a.o0) + t * a.ldo0 + c0, y);
    }
    const int s = REV ? s_start[k] : s_end[k];
    if (s >= 0 && a.out) Raw<float, V>::put(a.out + (long long)s * a.D + c0, y);
  }
}

// Before the scan: the sequences' first rows (lengths added up, each block all
// of those before its own: at most B / 1024 blocks read them from L2), the
// sequence of each chunk's first row, empty sequences' states (passed on), and
// the chain's flags zeroed.
struct PrepArgs {
  const int* lengths;  // null: only the flags, or every sequence is empty
  int *off, *first;
  int T, B, D, C, chunks;
  uint32_t* zero;
  long long zeros;
  const float* in;
  float* out;
  int* status;
};
constexpr int kPrep = 1024;
__global__ void __launch_bounds__(kPrep) prep_kernel(const __grid_constant__ PrepArgs a) {
  __shared__ long long part[kPrep / 32], before;
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_go();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * kPrep + tid; i < a.zeros; i += (long long)gridDim.x * kPrep) a.zero[i] = 0u;
  const long long s0 = (long long)blockIdx.x * kPrep;
  if (s0 >= a.B) return;
  const long long s = s0 + tid;
  int b = 0, e = 0;
  if (a.lengths) {
    if (tid == 0) bad = 0;
    long long sum = 0;
#pragma unroll 4
    for (long long i = tid; i < s0; i += kPrep) sum += max(__ldg(a.lengths + i), 0);
    const int raw = s < a.B ? __ldg(a.lengths + s) : 0, len = max(raw, 0);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      before = 0;
      for (int w = 0; w < kPrep / 32; ++w) before += part[w];
    }
    if (raw < 0) bad = 1;
    __syncthreads();
    long long end = len;  // inclusive, in the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long p = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += p;
    }
    if (lane == 31) part[warp] = end;
    __syncthreads();
    for (int w = 0; w < warp; ++w) end += part[w];
    end += before;
    const long long T = a.T;
    if (s == a.B - 1 && a.status && end > T) atomicOr(a.status, DSF_FLAG_COUNT);
    if (tid == 0 && bad && a.status) atomicOr(a.status, DSF_FLAG_NEG_LENGTH);
    b = int(min(end - len, T));
    e = int(min(end, T));
    if (s < a.B) {
      a.off[s] = b;
      if (s == a.B - 1) a.off[a.B] = e;
    }
    // chunks that begin in this sequence (many of a long one: by the warp)
    const int k0 = (b + a.C - 1) / a.C, k1 = e > b ? (e - 1) / a.C + 1 : k0;
    const bool many = s < a.B && k1 - k0 > 4;
    if (s < a.B && !many)
      for (int k = k0; k < k1; ++k) a.first[k] = int(s);
    for (uint32_t m = __ballot_sync(0xffffffffu, many); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const int j0 = __shfl_sync(0xffffffffu, k0, l), j1 = __shfl_sync(0xffffffffu, k1, l);
      for (int k = j0 + lane; k < j1; k += 32) a.first[k] = int(s0) + warp * 32 + l;
    }
  }
  if (!a.out) return;
  if (a.lengths || a.T == 0)  // (equal lengths: none is empty, or all are)
    for (uint32_t m = __ballot_sync(0xffffffffu, s < a.B && b == e); m; m &= m - 1) {
      const long long q = (s0 + warp * 32 + __ffs(m) - 1) * a.D;
      for (int c = lane; c < a.D; c += 32) a.out[q + c] = a.in ? a.in[q + c] : 0.f;
    }
}

// ---------------------------------------------------------------- host side
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool at(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Plan {
  int V, NT, log_ct, C, tiles;
  long long chunks, groups;
  size_t off, first, flags, pairs, states, total;  // flags: the ticket, the chunks', the groups'
};
Plan plan(long long T, long long B, int D, bool vec, bool rev) {
  Plan p{};
  p.V = vec ? 4 : 1;
  p.NT = rev ? kBwdRows : kFwdRows;
  const int most = vec ? 4 : 5, lanes = (D + p.V - 1) / p.V;  // threads along the channels: 4 .. 16 (32)
  p.log_ct = 2;
  while (p.log_ct < most && (1 << p.log_ct) < lanes) ++p.log_ct;
  p.C = (kThreads >> p.log_ct) * p.NT;
  const int width = (1 << p.log_ct) * p.V;
  p.tiles = (D + width - 1) / width;
  p.chunks = (T + p.C - 1) / p.C;
  p.groups = (p.chunks + kGroup - 1) / kGroup;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t here = o;
    o += align256(bytes);
    return here;
  };
  p.off = take(size_t(B + 1) * 4);
  p.first = take(size_t(p.chunks + 1) * 4);
  p.flags = take(size_t(1 + (p.chunks + p.groups) * p.tiles) * 4);
  p.pairs = take(size_t(p.chunks) * p.tiles * width * 8);
  p.states = take(size_t(p.groups) * p.tiles * width * 4);
  p.total = o;
  return p;
}

bool sizes_ok(int64_t T, int64_t B, int32_t D) {
  return T >= 0 && T <= kMaxRows && B >= 0 && B <= kMaxRows && D >= 1 && D <= kMaxDim;
}
size_t ws_bytes_of(int64_t T, int64_t B, int32_t D) {
  size_t most = 0;
  for (int i = 0; i < 4; ++i) {
    if ((i & 1) && D % 4) continue;
    const Plan p = plan(T, B, D, i & 1, i & 2);
    most = p.total > most ? p.total : most;
  }
  return most + 256;
}

template <class T, int V, int NT, bool REV>
bool launch(const Args& a, long long blocks, cudaStream_t s) {
  return pdl_launch(scan_kernel<T, V, NT, REV>, dim3(unsigned(blocks)), kThreads, s, a);
}

// rows of `es`-byte elements that vectors of four may be taken from
bool vec_rows(const void* p, long long ld, int es) { return !p || (at(p, 4 * es) && ld % 4 == 0); }

template <bool REV>
int run(Args a, int32_t dtype, const int32_t* lengths, uint8_t* ws, cudaStream_t s) {
  const int es = dtype == DSF_F32 ? 4 : 2;
  const bool vec = a.D % 4 == 0 && vec_rows(a.x, a.ldx, es) && vec_rows(a.gate, a.ldg, es) && vec_rows(a.h, a.ldh, es) &&
                   vec_rows(a.dh, a.lddh, es) && vec_rows(a.o0, a.ldo0, es) && vec_rows(a.o1, a.ldo1, es) && at(a.in, 16) &&
                   at(a.h0, 16) && at(a.out, 16);
  const Plan p = plan(a.T, a.B, a.D, vec, REV);
  if (p.chunks * p.tiles > INT32_MAX) return DSF_EUNSUPPORTED;
  a.chunks = int(p.chunks);
  a.tiles = p.tiles;
  a.log_ct = p.log_ct;
  a.L = a.B > 0 ? a.T / a.B : 0;
  a.off = lengths ? reinterpret_cast<int*>(ws + p.off) : nullptr;
  a.first = reinterpret_cast<int*>(ws + p.first);
  a.ticket = reinterpret_cast<uint32_t*>(ws + p.flags);
  a.flags = a.ticket + 1;
  a.group_flags = a.flags + p.chunks * p.tiles;
  a.pairs = reinterpret_cast<float2*>(ws + p.pairs);
  a.states = reinterpret_cast<float*>(ws + p.states);
  a.chain = p.chunks > 1 && (lengths || p.C % a.L != 0);
  if (lengths || a.chain || (a.T == 0 && a.out)) {
    PrepArgs q{lengths, reinterpret_cast<int*>(ws + p.off), reinterpret_cast<int*>(ws + p.first), a.T, a.B, a.D, p.C,
               int(p.chunks), a.ticket, a.chain ? 1 + (p.chunks + p.groups) * p.tiles : 0, a.in, a.out, a.status};
    long long blocks = (lengths || a.T == 0) ? ((long long)a.B + kPrep - 1) / kPrep : 1;
    const long long zeroing = (q.zeros + 8 * kPrep - 1) / (8 * kPrep), most = 152;
    if (blocks < zeroing) blocks = zeroing < most ? zeroing : (blocks < most ? most : blocks);
    if (!pdl_launch(prep_kernel, dim3(unsigned(blocks)), kPrep, s, q)) return DSF_ECUDA;
  }
  if (a.T == 0) return DSF_OK;
  constexpr int NT = REV ? kBwdRows : kFwdRows;
  const long long blocks = p.chunks * p.tiles;
  const bool ok = dtype == DSF_F32
                      ? (vec ? launch<float, 4, NT, REV>(a, blocks, s) : launch<float, 1, NT, REV>(a, blocks, s))
                      : (vec ? launch<__nv_bfloat16, 4, NT, REV>(a, blocks, s) : launch<__nv_bfloat16, 1, NT, REV>(a, blocks, s));
  return ok ? DSF_OK : DSF_ECUDA;
}

// A [rows, D] matrix of es-byte elements with row stride ld
bool rows_ok(const void* p, int64_t ld, int32_t D, int es) { return p && ld >= D && at(p, es); }

int check(int32_t dtype, const int32_t* lengths, int64_t T, int32_t B, int32_t D, const float* s0, const float* s1,
          const float* s2) {
  if (dtype != DSF_F32 && dtype != DSF_BF16) return DSF_EUNSUPPORTED;
  if (!sizes_ok(T, B, D) || !at(lengths, 4) || !at(s0, 4) || !at(s1, 4) || !at(s2, 4)) return DSF_EINVAL;
  if (!lengths && B > 0 && T % B != 0) return DSF_EINVAL;
  return DSF_OK;
}
int check_ws(int64_t T, int32_t B, int32_t D, const void* ws, size_t ws_bytes) {
  return ws && at(ws, 256) && ws_bytes >= ws_bytes_of(T, B, D) ? DSF_OK : DSF_EWORKSPACE;
}

}  // namespace
}  // namespace scan
}  // namespace dsf

using namespace dsf::scan;

extern "C" {

size_t dsf_gated_scan_workspace_bytes(int64_t T, int32_t B, int32_t D) {
  return sizes_ok(T, B, D) ? ws_bytes_of(T, B, D) : 0;
}

int ctr_gated_scan_fwd(const void* x, int64_t ldx, const void* gate, int64_t ldg, int32_t dtype, const int32_t* lengths,
                       int64_t T, int32_t B, int32_t D, const float* h0, void* h, int64_t ldh, float* h_last, void* ws,
                       size_t ws_bytes, int32_t* status, void* stream) {
  if (int rc = check(dtype, lengths, T, B, D, h0, h_last, nullptr)) return rc;
  const int es = dtype == DSF_F32 ? 4 : 2;
  if (T > 0 && (!rows_ok(x, ldx, D, es) || !rows_ok(gate, ldg, D, es) || !rows_ok(h, ldh, D, es))) return DSF_EINVAL;
  if (int rc = check_ws(T, B, D, ws, ws_bytes)) return rc;
  if (B == 0) return DSF_OK;
  Args a{};
  a.x = x, a.ldx = ldx, a.gate = gate, a.ldg = ldg, a.o0 = h, a.ldo0 = ldh;
  a.in = h0, a.out = h_last;
  a.T = int(T), a.B = B, a.D = D, a.status = status;
  return run<false>(a, dtype, lengths, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
}

int ctr_gated_scan_bwd(const void* dh, int64_t lddh, const void* x, int64_t ldx, const void* gate, int64_t ldg,
                       const void* h, int64_t ldh, int32_t dtype, const int32_t* lengths, int64_t T, int32_t B, int32_t D,
                       const float* h0, const float* dh_last, void* dx, int64_t lddx, void* dgate, int64_t lddg,
                       float* dh0, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  if (int rc = check(dtype, lengths, T, B, D, h0, dh_last, dh0)) return rc;
  const int es = dtype == DSF_F32 ? 4 : 2;
  if (T > 0 && (!rows_ok(dh, lddh, D, es) || !rows_ok(x, ldx, D, es) || !rows_ok(gate, ldg, D, es) ||
                !rows_ok(h, ldh, D, es) || !rows_ok(dx, lddx, D, es) || !rows_ok(dgate, lddg, D, es)))
    return DSF_EINVAL;
  if (int rc = check_ws(T, B, D, ws, ws_bytes)) return rc;
  if (B == 0) return DSF_OK;
  Args a{};
  a.x = x, a.ldx = ldx, a.gate = gate, a.ldg = ldg, a.h = h, a.ldh = ldh, a.dh = dh, a.lddh = lddh;
  a.o0 = dx, a.ldo0 = lddx, a.o1 = dgate, a.ldo1 = lddg;
  a.in = dh_last, a.h0 = h0, a.out = dh0;
  a.T = int(T), a.B = B, a.D = D, a.status = status;
  return run<true>(a, dtype, lengths, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
