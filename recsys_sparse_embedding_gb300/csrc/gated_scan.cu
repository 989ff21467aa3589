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
// One pass over memory. An item is a chunk of rows by up to 32 channels (a
// thread: 4 channels by NT rows, in registers as what each row is without the
// state before the thread's rows and what that state is multiplied with). The
// item's pair is published at once; its state is then put together from the
// pairs of the chunks before it, and its rows are written. (Without that, a pass
// for the pairs and a second over x and gate would move 5/3 of the bytes.) Blocks
// are persistent: as soon as an item's rows are in registers, the next item's are
// on their way to shared memory (cp.async, each thread what it will use itself).
// Blocks take items by a ticket, so they only wait for blocks that have started,
// whatever else runs; every wait is bounded and sets DSF_FLAG_TIMEOUT when it
// runs out.
//
// Fixed order: chunks are in groups (8 of 32 channels, 16 of 16: a pair per thread); a
// chunk starts from the state at the end of the group before its own and composes the
// pairs of its group in a fixed tree, so equal calls give equal bits, however blocks are scheduled, and
// the chain through memory has one step per group. A pair and a state are 8
// bytes, stored and polled whole; all bits set means "not there yet" (no
// arithmetic gives that NaN), so no flag and no fence is needed.
//
// A reset is carried as A = -1 (A is never negative otherwise): nothing is
// multiplied across a sequence's border, so a non-finite state stays in its
// own sequence. States, pairs and sums are fp32; h, dx and dgate are rounded
// once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "dense_math.cuh"
#include "dinsparse.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace dsf {
namespace scan {
namespace {

constexpr int kSms = 152;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostWidth = 32;  // channels of an item
constexpr int kMaxDim = 1 << 20;
constexpr long long kMaxRows = 1 << 30, kMaxSequences = 1 << 26;  // (sequences that have lengths)

// rows per thread (the backward keeps four values of each element, the forward two)
template <class T, bool REV>
constexpr int rows_of() {
  return REV ? 4 : 8;
}

struct Args {
  const void *x, *gate, *h, *dh;  // h, dh: backward
  void *o0, *o1;                  // h; dx and dgate
  long long ldx, ldg, ldh, lddh, ldo0, ldo1;
  const float* in;  // [B, D]: h0; dh_last (nullable)
  const float* h0;  // backward: [B, D] (nullable)
  float* out;       // [B, D]: h_last; dh0 (nullable)
  const int* total;           // rows of all sequences; null: T, equal lengths L
  const uint8_t* mark;        // per row: 1 a sequence's first, 2 its last
  const int *first, *last;    // the sequence of such a row (other entries hold nothing)
  int T, D, L;
  int tiles;
  int chain;  // whether a sequence may go on from chunk to chunk
  uint32_t* ticket;           // one less than the next item
  unsigned long long* pairs;  // [chunks][tiles][4 CT]
  unsigned long long* states; // [groups][tiles][4 CT]: a state, and 0
  int* status;
};

// four neighbouring elements of a row
template <class T>
struct Raw;
template <>
struct Raw<float> {
  uint4 v;
  __device__ void get(float2* f) const {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ void set(const float2* f) {
    v = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 v;
  __device__ void get(float2* f) const {
    f[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
  __device__ void set(const float2* f) { v = make_uint2(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y)); }
};
// n (0 .. 4) elements from p, the others zero; any alignment
template <class T>
__device__ __forceinline__ void load_few(Raw<T>& r, const T* p, int n) {
  float2 f[2] = {};
  if (n > 0) f[0].x = float(p[0]);
  if (n > 1) f[0].y = float(p[1]);
  if (n > 2) f[1].x = float(p[2]);
  if (n > 3) f[1].y = float(p[3]);
  r.set(f);
}
template <bool VEC, class T>
__device__ __forceinline__ void store4(T* p, const float2* f, int n) {
  if (VEC) {
    Raw<T> r;
    r.set(f);
    *reinterpret_cast<decltype(r.v)*>(p) = r.v;
    return;
  }
  if (n > 0) p[0] = T(f[0].x);
  if (n > 1) p[1] = T(f[0].y);
  if (n > 2) p[2] = T(f[1].x);
  if (n > 3) p[3] = T(f[1].y);
}
template <bool VEC>
__device__ __forceinline__ void load_state(const float* p, float2* f, int n) {
  Raw<float> r;
  if (VEC) r.v = __ldg(reinterpret_cast<const uint4*>(p));
  else load_few(r, p, n);
  r.get(f);
}
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src, bool any) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES),
               "r"(any ? BYTES : 0)
               : "memory");
}

// z = sigmoid(g) and a = 1 - z, each to (8 + 2 |g|) 2^-23 of its own size (below 2^-126:
// 0); what grows with |g| is the exponent's rounding, as much as one of g itself. Where a
// is below a half it is t z, t = exp(-g). Above, that product would be up to 2^-23 off 1,
// alike in every row of a constant gate: a closed one lost or gained 2% of its state in
// 131,072 rows. 1 - z is rounded once, never passes 1, and is 1 where z is nothing beside
// it. (One reciprocal of a product for four channels, with a branch for far gates, was
// slower: the special functions do not bind, and the branch keeps the rows apart.)
__device__ __forceinline__ void gate_of(float2 g, float2& z, float2& a) {
  const float2 e = g * pair(-kLog2e), t = make_float2(exp2_fast(e.x), exp2_fast(e.y)), d = t + pair(1.f);
  z = make_float2(rcp_fast(d.x), rcp_fast(d.y));
  const float2 rest = __ffma2_rn(z, pair(-1.f), pair(1.f));
  a = t * z;
  if (t.x > 1.f) a.x = rest.x;
  if (t.y > 1.f) a.y = rest.y;
}

// (A, B) := (A, B) after (Ap, Bp)
__device__ __forceinline__ void compose(float Ap, float Bp, float& A, float& B) {
  if (A < 0.f) return;
  B = fmaf(A, Bp, B);
  A = Ap < 0.f ? -1.f : A * Ap;
}
__device__ __forceinline__ float apply(float A, float B, float y) { return A < 0.f ? B : fmaf(A, y, B); }

constexpr unsigned long long kNone = ~0ull;
// A pair or a state, once it is there; false after about a second.
__device__ __forceinline__ bool take(const unsigned long long* p, unsigned long long v, float2& f) {
  bool ok = true;
  if (v == kNone) {
    const uint64_t t0 = globaltimer_ns();
    while ((v = ld_relaxed_u64(p)) == kNone)
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        ok = false;
        break;
      }
  }
  f = make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
  return ok;
}
__device__ __forceinline__ void give(unsigned long long* p, float2 f) {
  st_relaxed_u64(p, uint64_t(__float_as_uint(f.y)) << 32 | __float_as_uint(f.x));
}

// What a warp's rows are: none a sequence's border; some; or not all of the chunk's
// rows are there.
enum { kPlain = 0, kMarked = 1, kPartial = 2 };
template <int K>
using Kind = std::integral_constant<int, K>;

template <class T, bool REV>
struct Shared {
  static constexpr int NT = rows_of<T, REV>(), NA = REV ? 4 : 2;
  static constexpr int kData = NA * NT * kThreads * int(sizeof(Raw<T>));
  static constexpr int kBytes = kData + 8 * kThreads;
};

template <class T, bool REV, bool VEC, int LOG_CT>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) scan_kernel(const __grid_constant__ Args a) {
  using S = Shared<T, REV>;
  constexpr int NT = S::NT, NA = S::NA;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ float2 s_pair[kWarps][kMostWidth];  // the warps' pairs, then those of the warps before
  __shared__ float2 s_look[kWarps * kMostWidth];
  __shared__ float s_carry[kMostWidth];
  __shared__ int s_comes, s_ticket;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int CT = 1 << LOG_CT, C = (kThreads >> LOG_CT) * NT, W = 4 * CT;
  constexpr int log_group = 6 - LOG_CT;  // chunks of a group: a pair per thread
  const int ct = tid & (CT - 1), slice = tid >> LOG_CT;
  pdl_go();
  pdl_wait();
  const int total = a.total ? *a.total : a.T, chunks = (total + C - 1) / C;
  const int items = chunks * a.tiles;  // (below 2^30: checked by the host)

  struct Item {
    int rank, tile, t0, n;  // n = 0: none
  };
  auto item_at = [&](int idx) {
    Item it{0, 0, 0, 0};
    if (idx >= items) return it;
    it.rank = int(uint32_t(idx) / uint32_t(a.tiles));
    it.tile = idx - it.rank * a.tiles;
    it.t0 = (REV ? chunks - 1 - it.rank : it.rank) * C;
    it.n = min(C, total - it.t0);
    return it;
  };
  // the thread's rows, in scan order: upwards, or from the chunk's end
  auto row_of = [&](int i) { return REV ? C - 1 - (slice * NT + i) : slice * NT + i; };
  const int low = REV ? C - NT - slice * NT : slice * NT;  // the lowest of them
  auto slot = [&](int arr, int i) { return reinterpret_cast<Raw<T>*>(sm) + (arr * NT + i) * kThreads + tid; };
  uint8_t* marks = sm + S::kData + 8 * tid;
  auto width = [&](const Item& it) { return a.D - (it.tile * CT + ct) * 4; };  // channels from the thread's first on

  // a chunk's rows that are all there (most are): the loops over them unrolled
  auto whole = [&](const Item& it) { return VEC && it.n == C && (!REV || it.t0 > 0); };

  auto load = [&](const Item& it) {
    const int c0 = (it.tile * CT + ct) * 4, w = min(4, width(it));
    const bool live = it.n > 0 && w > 0;
    if (live) {
      const T* src[4] = {static_cast<const T*>(a.x), static_cast<const T*>(a.gate), static_cast<const T*>(a.dh),
                         static_cast<const T*>(a.h)};
      const long long ld[4] = {a.ldx, a.ldg, a.lddh, a.ldh};
#pragma unroll
      for (int arr = 0; arr < NA; ++arr) {
        const long long t = it.t0 + low - (arr == 3 ? 1 : 0);  // h: the row before
        const T* p = src[arr] + t * ld[arr] + c0;
        Raw<T>* d = slot(arr, REV ? NT - 1 : 0);
        constexpr int kNext = REV ? -kThreads : kThreads;
        if (whole(it)) {
#pragma unroll
          for (int k = 0; k < NT; ++k, p += ld[arr]) cp_async<int(sizeof(Raw<T>))>(d + k * kNext, p, true);
        } else {
#pragma unroll 1
          for (int k = 0; k < NT; ++k, p += ld[arr], d += kNext) {
            const bool any = low + k < it.n && t + k >= 0;
            if (VEC) {
              cp_async<int(sizeof(Raw<T>))>(d, any ? p : src[arr], any);
            } else {
              Raw<T> r;
              load_few(r, p, any ? w : 0);
              *d = r;
            }
          }
        }
      }
      if (a.total) cp_async<NT>(marks, a.mark + it.t0 + low, true);
    }
    cp_async_commit();
    if (live && !a.total) {
      int r = (it.t0 + low) % a.L;
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        marks[k] = uint8_t((r == 0 ? 1 : 0) | (r == a.L - 1 ? 2 : 0));
        r = r + 1 == a.L ? 0 : r + 1;
      }
    }
  };
  // the marks of the thread's rows as two sets of bits (bit i: row i in scan
  // order): where the recurrence starts anew, and where its state leaves
  auto sets = [&](const Item& it, uint32_t& reset, uint32_t& leave) {
    reset = leave = 0;
    const uint32_t m0 = *reinterpret_cast<const uint32_t*>(marks),
                   m1 = NT == 8 ? *reinterpret_cast<const uint32_t*>(marks + 4) : 0;
    if (!(m0 | m1)) return;
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const uint32_t b = low + k < it.n ? (k < 4 ? m0 : m1) >> (8 * (k & 3)) & 3u : 0u;
      const int i = REV ? NT - 1 - k : k;
      reset |= ((REV ? b >> 1 : b) & 1u) << i;
      leave |= ((REV ? b : b >> 1) & 1u) << i;
    }
  };
  auto seq_first = [&](long long t) { return a.total ? a.first[t] : int(t / a.L); };
  auto seq_last = [&](long long t) { return a.total ? a.last[t] : int(t / a.L); };

  // The thread's rows in scan order. Forward: h = u[0] + u[1] y with y the state
  // before them; backward: dx = u[0] + u[1] y, dgate = u[2] + u[3] y.
  constexpr int NU = REV ? 4 : 2;
  float2 u[NT][NU][2];
  float2 A[2], Bv[2];  // the thread's pair
  float2 leaveA[2], leaveB[2];  // backward: that of the rows up to the first that leaves, if no reset is among them
  uint32_t reset, leave;
  auto rows = [&](const Item& it, auto kind) {
    constexpr bool PLAIN = kind == kPlain, WHOLE = kind != kPartial;
    const int c0 = (it.tile * CT + ct) * 4;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (!WHOLE && row_of(i) >= it.n) continue;
      float2 g[2], v[2], z[2], a1[2], x[2], hp[2];
      slot(1, i)->get(g);
      slot(REV ? 2 : 0, i)->get(v);
      if (REV) {
        slot(0, i)->get(x);
        slot(3, i)->get(hp);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) gate_of(g[h], z[h], a1[h]);
      if (!PLAIN) {
        const long long t = it.t0 + row_of(i);
        if (reset >> i & 1u) {
#pragma unroll
          for (int h = 0; h < 2; ++h) A[h] = Bv[h] = pair(0.f);
          if (a.in) {
            load_state<VEC>(a.in + (long long)(REV ? seq_last(t) : seq_first(t)) * a.D + c0, Bv, width(it));
          }
        }
        if (REV && (leave >> i & 1u)) {
          hp[0] = hp[1] = pair(0.f);
          if (a.h0) load_state<VEC>(a.h0 + (long long)seq_first(t) * a.D + c0, hp, width(it));
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (REV) {
          const float2 w = __ffma2_rn(hp[h], pair(-1.f), x[h]) * (z[h] * a1[h]), s = v[h] + Bv[h];
          u[i][0][h] = z[h] * s;
          u[i][1][h] = z[h] * A[h];
          u[i][NU - 2][h] = w * s;
          u[i][NU - 1][h] = w * A[h];
          Bv[h] = a1[h] * s;
          A[h] = a1[h] * A[h];
          if (!PLAIN && (leave >> i & 1u) && !(reset & ((2u << i) - 1))) leaveA[h] = A[h], leaveB[h] = Bv[h];
        } else {
          Bv[h] = __ffma2_rn(a1[h], Bv[h], z[h] * v[h]);
          A[h] = A[h] * a1[h];
          u[i][0][h] = Bv[h];
          u[i][1][h] = A[h];
        }
      }
      if (!PLAIN && REV && (leave >> i & 1u) && (reset & ((2u << i) - 1)) && a.out)
        store4<VEC>(a.out + (long long)seq_first(it.t0 + row_of(i)) * a.D + c0, Bv, width(it));
    }
  };
  // the rows' outputs, and the states that leave: those of the pair's last row y
  // steps on by
  auto write = [&](const Item& it, const float2* y, auto kind) {
    constexpr bool PLAIN = kind == kPlain, WHOLE = kind != kPartial;
    const int c0 = (it.tile * CT + ct) * 4, w = width(it);
    const long long t1 = it.t0 + row_of(0), d0 = REV ? -a.ldo0 : a.ldo0, d1 = -a.ldo1;
    T* o0 = static_cast<T*>(a.o0) + t1 * a.ldo0 + c0;
    T* o1 = REV ? static_cast<T*>(a.o1) + t1 * a.ldo1 + c0 : nullptr;
    const int first = PLAIN || !reset ? NT : __ffs(reset) - 1;  // (from there on y has no part)
#pragma unroll
    for (int i = 0; i < NT; ++i, o0 += d0, o1 += REV ? d1 : 0) {
      if (!WHOLE && row_of(i) >= it.n) continue;
      float2 p[2], q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        p[h] = __ffma2_rn(u[i][1][h], y[h], u[i][0][h]);
        if (REV) q[h] = __ffma2_rn(u[i][NU - 1][h], y[h], u[i][NU - 2][h]);
      }
      if (!PLAIN && i >= first) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          p[h] = u[i][0][h];
          if (REV) q[h] = u[i][NU - 2][h];
        }
      }
      store4<VEC>(o0, p, w);
      if (REV) store4<VEC>(o1, q, w);
      if (!PLAIN && !REV && (leave >> i & 1u) && a.out)
        store4<VEC>(a.out + (long long)seq_last(it.t0 + row_of(i)) * a.D + c0, p, w);
    }
    if (!PLAIN && REV && leave && !(reset & ((leave & -leave) * 2 - 1)) && a.out) {
      float2 p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) p[h] = __ffma2_rn(leaveA[h], y[h], leaveB[h]);
      store4<VEC>(a.out + (long long)seq_first(it.t0 + row_of(__ffs(leave) - 1)) * a.D + c0, p, w);
    }
  };

  int idx = blockIdx.x;
  uint32_t drawn = 0;  // (thread 0)
  auto request = [&]() {
    if (!a.chain) idx += gridDim.x;
    else if (tid == 0) drawn = atomicAdd(a.ticket, 1u) + 1u;
  };
  auto announce = [&]() {
    if (a.chain && tid == 0) s_ticket = int(min(drawn, uint32_t(items)));
    __syncthreads();
    if (a.chain) idx = s_ticket;
  };
  if (a.chain) {
    request();
    announce();
    __syncthreads();
  }
  bool ok = true;
  Item cur = item_at(idx);
  load(cur);
  while (cur.n > 0) {
    request();
    // the pairs of the item's group before it and the state before the group (looked
    // at now, awaited when the item's own pair is out)
    const int group = cur.rank >> log_group, j0 = (group << log_group) + tid / W;
    const long long step = (long long)a.tiles * W;
    const unsigned long long* pp = a.pairs + ((long long)j0 * a.tiles + cur.tile) * W + (tid & (W - 1));
    const unsigned long long* ps = a.states + ((long long)(group - 1) * a.tiles + cur.tile) * W + tid;
    unsigned long long raw = kNone, raw_state = kNone;
    const bool mine = a.chain && j0 < cur.rank;
    if (mine) raw = ld_relaxed_u64(pp);
    if (a.chain && group > 0 && tid < W) raw_state = ld_relaxed_u64(ps);

    cp_async_wait_all();
    const bool live = width(cur) > 0;
    A[0] = A[1] = pair(1.f);
    Bv[0] = Bv[1] = pair(0.f);
    reset = leave = 0;
    if (live) sets(cur, reset, leave);
    const int kind = whole(cur) ? (__any_sync(0xffffffffu, reset | leave) ? kMarked : kPlain) : kPartial;  // (the warp's: one way for all)
    if (live) {
      if (kind == kPlain) rows(cur, Kind<kPlain>{});
      else if (kind == kMarked) rows(cur, Kind<kMarked>{});
      else rows(cur, Kind<kPartial>{});
    }
    if (tid == 0) s_comes = a.chain && !(reset & 1u) && !(REV && cur.n < C);
    float qa[4] = {A[0].x, A[0].y, A[1].x, A[1].y}, qb[4] = {Bv[0].x, Bv[0].y, Bv[1].x, Bv[1].y};
    if (reset) qa[0] = qa[1] = qa[2] = qa[3] = -1.f;
    for (int d = CT; d < 32; d <<= 1)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float ap = __shfl_up_sync(0xffffffffu, qa[v], d), bp = __shfl_up_sync(0xffffffffu, qb[v], d);
        if (lane >= d) compose(ap, bp, qa[v], qb[v]);
      }
    if (lane >= 32 - CT)
#pragma unroll
      for (int v = 0; v < 4; ++v) s_pair[warp][ct * 4 + v] = make_float2(qa[v], qb[v]);
    announce();
    const bool comes = s_comes;
    const Item nxt = item_at(idx);
    load(nxt);  // (in the place that the thread has just read)
    float2 tot = make_float2(1.f, 0.f);  // (tid < W) the item's pair in channel tid
    if (tid < W) {
      float2 p[kWarps];
#pragma unroll
      for (int k = 0; k < kWarps; ++k) p[k] = s_pair[k][tid];
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        s_pair[k][tid] = tot;
        compose(tot.x, tot.y, p[k].x, p[k].y);
        tot = p[k];
      }
      if (a.chain) give(a.pairs + ((long long)cur.rank * a.tiles + cur.tile) * W + tid, tot);
    }
    if (comes) {
      float2 f = make_float2(1.f, 0.f);
      if (mine) ok = take(pp, raw, f) && ok;
      for (int d = W; d < 32; d <<= 1) {  // (the warp's pairs)
        const float ap = __shfl_up_sync(0xffffffffu, f.x, d), bp = __shfl_up_sync(0xffffffffu, f.y, d);
        if (lane >= d) compose(ap, bp, f.x, f.y);
      }
      if (lane >= 32 - W) s_look[warp * W + (lane & (W - 1))] = f;
      __syncthreads();
    }
    if (tid < W) {
      float y = 0.f;
      if (comes) {
        float QA = 1.f, QB = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          float2 f = s_look[k * W + tid];
          compose(QA, QB, f.x, f.y);
          QA = f.x, QB = f.y;
        }
        if (QA >= 0.f && group > 0) {
          float2 f;
          ok = take(ps, raw_state, f) && ok;
          y = f.x;
        }
        y = apply(QA, QB, y);
      }
      s_carry[tid] = y;
      if (a.chain && ((cur.rank + 1) & ((1 << log_group) - 1)) == 0) give(const_cast<unsigned long long*>(ps) + step, make_float2(apply(tot.x, tot.y, y), 0.f));
    }
    // the state before the thread's rows: of the warp's threads before it, of the warps
    // before, of the chunks before
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float ap = __shfl_up_sync(0xffffffffu, qa[v], CT), bp = __shfl_up_sync(0xffffffffu, qb[v], CT);
      qa[v] = lane >= CT ? ap : 1.f;
      qb[v] = lane >= CT ? bp : 0.f;
    }
    __syncthreads();
    if (live) {
      float2 y[2];
      float* yf = reinterpret_cast<float*>(y);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float2 e = s_pair[warp][ct * 4 + v];
        yf[v] = apply(qa[v], qb[v], apply(e.x, e.y, s_carry[ct * 4 + v]));
      }
      if (kind == kPlain) write(cur, y, Kind<kPlain>{});
      else if (kind == kMarked) write(cur, y, Kind<kMarked>{});
      else write(cur, y, Kind<kPartial>{});
    }
    cur = nxt;
  }
  if (!ok && a.status) atomicOr(a.status, DSF_FLAG_TIMEOUT);
}

// A step of serving: every sequence has one row, and nothing to be put together
// (512 x 256 bf16: 2.1 us in a graph; as a chunk of the scan 8.2).
template <class T, bool VEC>
__global__ void __launch_bounds__(256) step_kernel(const __grid_constant__ Args a) {
  pdl_go();
  pdl_wait();
  const int n4 = (a.D + 3) / 4;
  const long long i = blockIdx.x * 256LL + threadIdx.x, t = i / n4;
  if (t >= a.T) return;
  const int c0 = int(i - t * n4) * 4, w = a.D - c0;
  const T *px = static_cast<const T*>(a.x) + t * a.ldx + c0, *pg = static_cast<const T*>(a.gate) + t * a.ldg + c0;
  Raw<T> rx, rg;
  float2 x[2], g[2], h[2] = {pair(0.f), pair(0.f)};
  if (VEC) {
    rx.v = __ldg(reinterpret_cast<const decltype(rx.v)*>(px));
    rg.v = __ldg(reinterpret_cast<const decltype(rg.v)*>(pg));
  } else {
    load_few(rx, px, w);
    load_few(rg, pg, w);
  }
  if (a.in) load_state<VEC>(a.in + t * a.D + c0, h, w);
  rx.get(x);
  rg.get(g);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2 z, keep;
    gate_of(g[k], z, keep);
    h[k] = __ffma2_rn(keep, h[k], z * x[k]);
  }
  store4<VEC>(static_cast<T*>(a.o0) + t * a.ldo0 + c0, h, w);
  if (a.out) store4<VEC>(a.out + t * a.D + c0, h, w);
}

// Before the scan: the sequences' borders (lengths added up, each block all of
// those before its own, from L2; of very many sequences the sums of a block's
// lengths, which sums_kernel leaves) as marks on their rows, empty sequences' states
// (passed on), and the chain's pairs and ticket set to "not there".
struct PrepArgs {
  const int* lengths;  // null: no marks
  long long* sums;     // of 1024 lengths each (nullable)
  uint8_t* mark;
  int *first, *last, *total;
  int T, B, D;
  bool clear;  // whether the marks have to be set to 0 first
  uint4* fill;
  long long fills;
  const float* in;
  float* out;
  uint32_t* ticket;
  int* status;
};
constexpr int kPrep = 1024;
constexpr int kManySequences = 1 << 16;  // (the 8 MB that 64 blocks then read in all take less than a launch)
__global__ void __launch_bounds__(kPrep) sums_kernel(const int* lengths, int B, long long* sums) {
  __shared__ long long part[kPrep / 32];
  pdl_go();
  pdl_wait();
  const long long s = (long long)blockIdx.x * kPrep + threadIdx.x;
  long long n = s < B ? max(__ldg(lengths + s), 0) : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  n = part[threadIdx.x];
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (threadIdx.x == 0) sums[blockIdx.x] = n;
}
__global__ void __launch_bounds__(kPrep) prep_kernel(const __grid_constant__ PrepArgs a) {
  __shared__ long long part[kPrep / 32], before, after;
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_go();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * kPrep + tid; i < a.fills; i += (long long)gridDim.x * kPrep)
    a.fill[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  if (blockIdx.x == 0 && tid == 0) *a.ticket = ~0u;
  const long long s0 = (long long)blockIdx.x * kPrep;
  if (s0 >= a.B) return;
  const long long s = s0 + tid;
  int b = 0, e = 0;
  if (a.lengths) {
    if (tid == 0) bad = 0;
    long long sum = 0;
    if (a.sums) {
      for (int i = tid; i < int(blockIdx.x); i += kPrep) sum += a.sums[i];
    } else {
#pragma unroll 8
      for (long long i = tid; i < s0; i += kPrep) sum += max(__ldg(a.lengths + i), 0);
    }
    const int raw = s < a.B ? __ldg(a.lengths + s) : 0, len = max(raw, 0);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      sum = part[lane];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) before = sum;
    }
    if (raw < 0) bad = 1;
    long long end = len;  // inclusive, in the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long p = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += p;
    }
    __syncthreads();
    if (lane == 31) part[warp] = end;
    __syncthreads();
    long long ahead = lane < warp ? part[lane] : 0;  // of the warps before
#pragma unroll
    for (int o = 16; o; o >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    end += ahead + before;
    const long long T = a.T;
    if (a.clear) {  // the rows of the block's sequences
      if (tid == kPrep - 1) after = end;
      __syncthreads();
      const long long lo = min(before, T), hi = min(after, T), lo16 = min((lo + 15) & ~15LL, hi), hi16 = max(hi & ~15LL, lo16);
      if (tid < lo16 - lo) a.mark[lo + tid] = 0;
      for (long long i = lo16 + 16 * tid; i < hi16; i += 16 * kPrep) *reinterpret_cast<uint4*>(a.mark + i) = make_uint4(0, 0, 0, 0);
      if (tid < hi - hi16) a.mark[hi16 + tid] = 0;
      __syncthreads();
    }
    if (s == a.B - 1 && a.status && end > T) atomicOr(a.status, DSF_FLAG_COUNT);
    if (tid == 0 && bad && a.status) atomicOr(a.status, DSF_FLAG_NEG_LENGTH);
    b = int(min(end - len, T));
    e = int(min(end, T));
    if (s == a.B - 1) *a.total = e;
    if (s < a.B && e > b) {  // (the others are zero)
      a.first[b] = int(s);
      a.last[e - 1] = int(s);
      a.mark[b] = e - b == 1 ? 3 : 1;
      if (e - b > 1) a.mark[e - 1] = 2;
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

constexpr int rows_per_thread(int es, bool rev) {
  return es == 4 ? (rev ? rows_of<float, true>() : rows_of<float, false>())
                 : (rev ? rows_of<__nv_bfloat16, true>() : rows_of<__nv_bfloat16, false>());
}

struct Plan {
  int D, log_ct, C, tiles;
  long long chunks, groups;
  size_t mark, first, last, sync, sync_bytes, total;  // sync: the ticket and total, pairs, states
  size_t pairs, states, sums;
};
Plan plan(long long T, long long B, int D, int nt, int log_ct) {
  Plan p{};
  p.D = D;
  p.log_ct = log_ct;
  p.C = (kThreads >> p.log_ct) * nt;
  const int width = 4 << p.log_ct;
  p.tiles = (D + width - 1) / width;
  p.chunks = (T + p.C - 1) / p.C;
  p.groups = ((p.chunks - 1) >> (6 - p.log_ct)) + 1;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t here = o;
    o += align256(bytes);
    return here;
  };
  p.mark = take(size_t(p.chunks) * p.C);
  p.first = take(size_t(T) * 4);
  p.last = take(size_t(T) * 4);
  p.sync = take(256);
  p.pairs = take(size_t(p.chunks) * p.tiles * width * 8);
  p.states = take(size_t(p.groups) * p.tiles * width * 8);
  p.sync_bytes = o - p.sync;
  p.sums = take(B > kManySequences ? size_t((B + kPrep - 1) / kPrep) * 8 : 0);
  p.total = o;
  return p;
}

bool sizes_ok(int64_t T, int64_t B, int32_t D) {
  return T >= 0 && T <= kMaxRows && B >= 0 && B <= kMaxRows && D >= 1 && D <= kMaxDim;
}
// Threads of 4 channels side by side, as a power of two: 8; 4 where that leaves fewer
// without a channel, or where the chain binds: a group of 8 x 8 chunks' rows takes 0.55
// us, unless other sequences' are under way beside it, and the bytes move at 3.2 TB/s.
// (Chunks of 16 channels are longer in rows, and 16 of them are a group. Forward and
// backward with 8 | 4 | 2 threads, bf16, us: one sequence of 262,144 x 64 207 | 188 | 205,
// 64 of them 166 | 171 | 195; 131,071 x 1024 652 | 766 | 1084.)
int pick_ct(const Plan& p, long long B, size_t bytes) {
  if (p.tiles * 2 != (p.D + 15) / 16) return 2;
  const double window = 2.0 * kSms / p.tiles, chunks = double(p.chunks) / double(B), beside = chunks < window ? window / chunks : 1;
  return double(p.groups) * 0.55 / beside > double(bytes) / 3.2e6 ? 2 : 3;
}
size_t ws_bytes_of(int64_t T, int32_t B, int32_t D) {
  size_t most = 0;
  for (int log_ct = 2; log_ct < 4; ++log_ct)
    for (int nt = 4; nt <= 8; nt += 4) {
      const size_t n = plan(T, B, D, nt, log_ct).total;
      most = most > n ? most : n;
    }
  return most + 256;
}

template <class T, bool REV, bool VEC, int LOG_CT>
bool launch(const Args& a, long long items, cudaStream_t s) {
  using S = Shared<T, REV>;
  auto* kernel = scan_kernel<T, REV, VEC, LOG_CT>;
  static std::atomic<int> most[64];  // (host threads may race on it: each computes the same value)
  int dev = 0;
  if (!succeeded(cudaGetDevice(&dev)) || dev < 0 || dev >= 64) return false;
  int blocks = most[dev].load(std::memory_order_acquire);
  if (blocks == 0) {
    int sms = 0, per = 0;
    if (!succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes)) ||
        !succeeded(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) ||
        !succeeded(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, S::kBytes)) || per < 1)
      return false;
    blocks = sms * per;
    most[dev].store(blocks, std::memory_order_release);
  }
  return pdl_launch_smem(kernel, dim3(unsigned(items < blocks ? items : blocks)), kThreads, S::kBytes, s, a);
}

// rows of `es`-byte elements that vectors of four may be taken from
bool vec_rows(const void* p, long long ld, int es) { return !p || (at(p, 4 * es) && ld % 4 == 0); }

template <bool REV>
int run(Args a, int B, int32_t dtype, const int32_t* lengths, uint8_t* ws, cudaStream_t s) {
  const int es = dtype == DSF_F32 ? 4 : 2;
  const bool vec = a.D % 4 == 0 && vec_rows(a.x, a.ldx, es) && vec_rows(a.gate, a.ldg, es) && vec_rows(a.h, a.ldh, es) &&
                   vec_rows(a.dh, a.lddh, es) && vec_rows(a.o0, a.ldo0, es) && vec_rows(a.o1, a.ldo1, es) && at(a.in, 16) &&
                   at(a.h0, 16) && at(a.out, 16);
  if (!REV && !lengths && a.T == B && a.T > 0) {
    const long long threads = (long long)a.T * ((a.D + 3) / 4);
    if (threads > (long long)INT32_MAX * 256) return DSF_EUNSUPPORTED;
    const dim3 grid(unsigned((threads + 255) / 256));
    const bool ok = dtype == DSF_F32 ? (vec ? pdl_launch(step_kernel<float, true>, grid, 256, s, a)
                                            : pdl_launch(step_kernel<float, false>, grid, 256, s, a))
                                     : (vec ? pdl_launch(step_kernel<__nv_bfloat16, true>, grid, 256, s, a)
                                            : pdl_launch(step_kernel<__nv_bfloat16, false>, grid, 256, s, a));
    return ok ? DSF_OK : DSF_ECUDA;
  }
  const int nt = rows_per_thread(es, REV);
  Plan p = plan(a.T, B, a.D, nt, 3);
  if (pick_ct(p, B, size_t(a.T) * a.D * es * (REV ? 6 : 3)) == 2) p = plan(a.T, B, a.D, nt, 2);
  a.tiles = p.tiles;
  a.L = a.T / B;
  a.ticket = reinterpret_cast<uint32_t*>(ws + p.sync);
  int* total = reinterpret_cast<int*>(ws + p.sync) + 32;
  a.total = lengths ? total : nullptr;
  a.mark = ws + p.mark;
  a.first = reinterpret_cast<int*>(ws + p.first);
  a.last = reinterpret_cast<int*>(ws + p.last);
  a.pairs = reinterpret_cast<unsigned long long*>(ws + p.pairs);
  a.states = reinterpret_cast<unsigned long long*>(ws + p.states);
  a.chain = p.chunks > 1 && (lengths || p.C % a.L != 0);
  if (p.chunks * p.tiles > INT32_MAX / 2) return DSF_EUNSUPPORTED;
  if (lengths || a.chain || (a.T == 0 && a.out)) {
    long long* sums = lengths && B > kManySequences ? reinterpret_cast<long long*>(ws + p.sums) : nullptr;
    // the marks: each block its sequences' rows (one may have all of them), or a launch of its own
    const long long parts = ((long long)B + kPrep - 1) / kPrep;
    const bool clear = a.T <= (1 << 17) * (parts < 4 ? parts : 4);
    PrepArgs q{lengths, sums, ws + p.mark, const_cast<int*>(a.first), const_cast<int*>(a.last), total, a.T, B, a.D, clear,
               reinterpret_cast<uint4*>(ws + p.pairs), a.chain ? (long long)((p.sync_bytes - 256) / 16) : 0, a.in, a.out, a.ticket, a.status};
    long long blocks = (lengths || a.T == 0) ? ((long long)B + kPrep - 1) / kPrep : 1;
    const long long filling = (q.fills + 4 * kPrep - 1) / (4 * kPrep), most = kSms;
    if (blocks < filling) blocks = filling < most ? filling : (blocks < most ? most : blocks);
    if (lengths && !clear && !succeeded(cudaMemsetAsync(ws + p.mark, 0, size_t(a.T), s))) return DSF_ECUDA;
    if (sums && !pdl_launch(sums_kernel, dim3(unsigned(((long long)B + kPrep - 1) / kPrep)), kPrep, s, lengths, B, sums))
      return DSF_ECUDA;
    if (!pdl_launch(prep_kernel, dim3(unsigned(blocks)), kPrep, s, q)) return DSF_ECUDA;
  }
  if (a.T == 0) return DSF_OK;
  const long long items = p.chunks * p.tiles;
  auto any = [&](auto type, auto vectors) {
    using T = decltype(type);
    constexpr bool VEC = decltype(vectors)::value;
    return p.log_ct == 3 ? launch<T, REV, VEC, 3>(a, items, s) : launch<T, REV, VEC, 2>(a, items, s);
  };
  const bool ok = dtype == DSF_F32 ? (vec ? any(float(), std::true_type{}) : any(float(), std::false_type{}))
                                   : (vec ? any(__nv_bfloat16(), std::true_type{}) : any(__nv_bfloat16(), std::false_type{}));
  return ok ? DSF_OK : DSF_ECUDA;
}

// A [rows, D] matrix of es-byte elements with row stride ld
bool rows_ok(const void* p, int64_t ld, int32_t D, int es) { return p && ld >= D && at(p, es); }

int check(int32_t dtype, const int32_t* lengths, int64_t T, int32_t B, int32_t D, const float* s0, const float* s1,
          const float* s2) {
  if (dtype != DSF_F32 && dtype != DSF_BF16) return DSF_EUNSUPPORTED;
  if (!sizes_ok(T, B, D) || !at(lengths, 4) || !at(s0, 4) || !at(s1, 4) || !at(s2, 4)) return DSF_EINVAL;
  if (!lengths && B > 0 && T % B != 0) return DSF_EINVAL;
  if (lengths && B > kMaxSequences) return DSF_EUNSUPPORTED;
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
  a.T = int(T), a.D = D, a.status = status;
  return run<false>(a, B, dtype, lengths, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
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
  a.T = int(T), a.D = D, a.status = status;
  return run<true>(a, B, dtype, lengths, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
