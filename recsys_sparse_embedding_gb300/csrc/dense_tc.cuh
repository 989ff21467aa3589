// The matrix products of the dense operators on the tensor cores: D = A B^T
// with the operator's epilogue, sums in fp32.
//
// One persistent, warp-specialised kernel. A work unit is a tile of 128 CG x
// BN accumulators (CG CTAs of a cluster work on one tile together: CG = 2
// halves what each SM has to read of B), over all of K or one K-split.
//   warp 8   brings A and B by TMA: K-blocks of 128 bytes per row in the
//            128-byte swizzle, through a ring of stages;
//   warp 9   issues the MMAs (tcgen05.mma, in the cluster's first CTA) into
//            one of two accumulators in tensor memory;
//   warps 0-7 run the epilogue of the other accumulator: 32 rows (a warp's
//            lane quarter) by 128 bytes of output at a time, one row per lane.
//            Inputs (the residual, or the upstream gradient) and outputs pass
//            through a 4 KB buffer per item by TMA, two items ahead, so that
//            global memory sees whole rows of 128 bytes; a matrix whose rows
//            are not at 16-byte boundaries is copied by the warp instead.
// So a tile's loads, MMAs and epilogue overlap the next tile's. Operands come
// as three-dimensional tensors [plane][row][column]:
//   - K-major (columns are K) or MN-major (rows are K: W in dx = dz W, both
//     operands in dW = dz^T x, which needs no transposed copies);
//   - planes: the three bf16 terms of an fp32 operand (Terms below), and the
//     gate and up halves of a gated layer. A product runs over a list of
//     plane pairs (segments) into one accumulator.
//
// Terms: x = x1 + x2 + x3 exactly, each the leading 8 significant bits of what
// is left. x y = sum of the terms' products; those below 2^-21 of it (x2 y3,
// x3 y2, x3 y3) are dropped. The tensor cores truncate each addition to the
// accumulator (measured: a run of n additions is low by about n 2^-25 of the
// sum), so an fp32 product (PROMOTE) keeps its runs short: the five smaller
// pairs, at most 2^-7 of the sum, share one run, x1 y1 takes a run of its own
// per 4 K-blocks (16 additions), and the epilogue warps add the runs up in
// registers, rounding to nearest. Tiles are half as wide for it.
//
// Every wait is bounded; one that runs out sets DSF_FLAG_TIMEOUT.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dense_math.cuh"
#include "dinsparse.h"
#include "ptx.cuh"

namespace dsf {
namespace dense {

// What the epilogue does with an accumulator.
enum Epi {
  kEpiFwd = 0,   // out = residual + act(z), or act(z) * z' for a gated layer
  kEpiDz = 1,    // out = dz (planes dg, du for a gated layer) from in = dy; column sums
  kEpiOut = 2,   // out = the accumulator
  kEpiPart = 3,  // fp32 partial sums of a K-split: plane split * planes + (half or batch)
};
enum Kind { kBf16 = 0, kE4m3 = 1 };
enum Major { kKK = 0, kKN = 1, kNN = 2 };  // A and B K-major; B MN-major; both

constexpr int kMaxSeg = 12;

struct TcArgs {
  int M, N;          // rows; output columns (a gated layer's: F)
  int mt, nt, nb;    // tiles along M and N, batches (halves of dW)
  int nkb, kbps;     // K-blocks per segment, per split
  int nbig;          // PROMOTE: the last nbig segments are the products of leading terms
  int splits, nseg;
  uint8_t pa[kMaxSeg], pb[kMaxSeg];  // the segments' planes (A: + batch; B of a gated layer: 2 pb, 2 pb + 1)
  int act;
  const float *bias, *xs, *ws;  // z = acc * xs[m] * ws[n] + bias[n] (each nullable; the up half at n + N)
  const void* in;
  long long ldi;
  int has_in, in_tma;
  void* out;
  long long ldo, out_plane;  // strides in elements
  int out_tma;
  float* part;  // kEpiDz: column sums of 32 rows each, [ceil(M / 32)][halves * N] (nullable)
  int* status;
};

// ---------------------------------------------------------------- inline PTX
template <int CG>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else  // (the barrier may be the other CTA's of the pair)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups have read their shared memory
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* slot, uint32_t cols) {
  if (CG == 1) tmem_alloc(slot, cols);
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_relinquish_cg() {
  if (CG == 1) tmem_relinquish();
  else asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t t, uint32_t cols) {
  if (CG == 1) tmem_dealloc(t, cols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}
template <int CG, int KIND>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
#define DSF_MMA(GROUP, K)                                                                                          \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::" GROUP ".kind::" K            \
               " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),                                                              \
               "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                                         \
               : "memory")
  if (KIND == kBf16) {
    if (CG == 1) DSF_MMA("1", "f16");
    else DSF_MMA("2", "f16");
  } else {
    if (CG == 1) DSF_MMA("1", "f8f6f4");
    else DSF_MMA("2", "f8f6f4");
  }
#undef DSF_MMA
}
// Arrives on the barrier (at this offset in each CTA of the cluster) once the
// thread's MMAs so far are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (CG == 1) tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
        : "memory");
}

// MN-major operand in the 128-byte swizzle: rows of 64 elements (one K index
// each), 8-row atoms of 1024 bytes along K (SBO), the next 64 elements along
// M or N 8 KB further (LBO).
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFFu) | uint64_t(8192u >> 4) << 16 | uint64_t(1024u >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}

// ---------------------------------------------------------------- shapes
template <int CG, int BN, bool GATED, int EPI>
struct Shape {
  static constexpr int kEpiWarps = 8, kThreads = 32 * (kEpiWarps + 2);
  static constexpr int BNC = BN / CG;            // B rows (or MN-major columns) in this CTA
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BNC * 128, STAGE = A_BYTES + B_BYTES;
  // item buffers per epilogue warp, 4 KB each
  static constexpr int NBUF = (EPI == kEpiFwd && !GATED) || EPI == kEpiDz ? 3 : 2;
  static constexpr int EBYTES = kEpiWarps * NBUF * 4096;
  static constexpr int kRoom = 227 * 1024 - 1024 - 512 - EBYTES;
  static constexpr int STAGES = kRoom / STAGE < 8 ? kRoom / STAGE : 8;
  static constexpr int SMEM = STAGES * STAGE + EBYTES + 512 + 1024;
  static constexpr uint32_t TCOLS = 2 * BN;      // two accumulators
  static_assert(TCOLS <= 512 && (TCOLS & (TCOLS - 1)) == 0, "tensor memory columns");
  static_assert(STAGES >= 3, "ring");
  static_assert(B_BYTES % (GATED && CG == 1 ? 2048 : 1024) == 0, "swizzle atoms");
};

struct Bars {
  uint64_t full[8], empty[8], tfull[2], tempty[2], in[8][3];
  uint32_t tmem;
  int abort_;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// sums of 32 columns over a warp's 32 rows (one row per lane): lane l returns
// column l's. Each step halves the columns a lane holds.
__device__ __forceinline__ float column_sum(float* v, int lane) {
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
    }
  }
  return v[0];
}

__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  tmem_ld16(t, v);
  tmem_ld16(t + 16, v + 16);
}

// n uniform fp32 values per lane (bias, scales): columns c .. c + 31 below N
__device__ __forceinline__ void load_cols(const float* p, int c, int N, bool vec, float* v) {
  if (vec && c + 32 <= N) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + c) + k);
      v[4 * k] = f.x, v[4 * k + 1] = f.y, v[4 * k + 2] = f.z, v[4 * k + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = c + k < N ? __ldg(p + c + k) : 0.f;
  }
}

template <int ACT, bool GATED>
__device__ __forceinline__ void act_fwd(float* g, const float* u) {
#pragma unroll
  for (int k = 0; k < 32; ++k) g[k] = GATED ? act_value<ACT>(g[k]) * u[k] : act_value<ACT>(g[k]);
}
// in d (the upstream gradient): g <- its dz; gated: g <- dg, u <- du
template <int ACT, bool GATED>
__device__ __forceinline__ void act_bwd(const float* d, float* g, float* u) {
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float2 f = act_both<ACT>(g[k]);
    if (GATED) {
      g[k] = d[k] * u[k] * f.y;
      u[k] = d[k] * f.x;
    } else {
      g[k] = d[k] * f.y;
    }
  }
}

// ---------------------------------------------------------------- the kernel
constexpr int kRun = 4;  // PROMOTE: K-blocks of leading terms per run

// Accumulator runs of a unit with kbn K-blocks per segment.
template <bool PROMOTE>
__device__ __forceinline__ int runs_of(const TcArgs& a, int kbn) {
  return PROMOTE ? (a.nseg > a.nbig ? 1 : 0) + (a.nbig * kbn + kRun - 1) / kRun : 1;
}

template <int CG, int BN, int MAJOR, int KIND, bool GATED, int EPI, class TO, bool PROMOTE>
__global__ void __launch_bounds__(Shape<CG, BN, GATED, EPI>::kThreads, 1)
    tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap mapA,
              const __grid_constant__ CUtensorMap mapB, const __grid_constant__ CUtensorMap mapI,
              const __grid_constant__ CUtensorMap mapO) {
  using S = Shape<CG, BN, GATED, EPI>;
  constexpr bool AMN = MAJOR == kNN, BMN = MAJOR != kKK;
  constexpr int kBK = KIND == kBf16 ? 64 : 128;            // K elements per block (128 bytes)
  constexpr int ON = GATED ? BN / 2 : BN;                  // output columns per tile
  constexpr int CW = 128 / int(sizeof(TO));                // output columns per item
  constexpr int NBUF = S::NBUF, STAGES = S::STAGES;
  static_assert(!(GATED && BMN), "a gated layer's product is K-major");
  extern __shared__ uint8_t dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* sE = sm + STAGES * S::STAGE;
  Bars* bars = reinterpret_cast<Bars*>(sE + S::EBYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int unit0 = blockIdx.x / CG, units_step = gridDim.x / CG;
  const int tiles = a.mt * a.nt * a.nb, units = tiles * a.splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->tfull[i], 1);
      mbar_init(&bars->tempty[i], S::kEpiWarps * CG);
    }
    for (int w = 0; w < S::kEpiWarps; ++w)
      for (int i = 0; i < 3; ++i) mbar_init(&bars->in[w][i], 1);
    bars->abort_ = 0;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc_cg<CG>(&bars->tmem, S::TCOLS);
    tmem_relinquish_cg<CG>();
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = bars->tmem;
  volatile int* aborted = &bars->abort_;

  // a unit: split-minor, then N tiles within groups of M tiles, so that the
  // units in flight share rows of A and of B in L2
  struct Unit {
    int m0, n0, batch, split, kb0, kbn;
  };
  auto unit_of = [&](int u) {
    Unit t;
    t.split = u % a.splits;
    int r = u / a.splits;
    const int per_b = a.mt * a.nt;
    t.batch = r / per_b;
    r -= t.batch * per_b;
    constexpr int G = 8;
    const int grp = r / (G * a.nt), first = grp * G, gm = min(G, a.mt - first);
    r -= grp * G * a.nt;
    t.m0 = (first + r % gm) * 128 * CG + int(rank) * 128;
    t.n0 = (r / gm) * ON;
    t.kb0 = t.split * a.kbps;
    t.kbn = min(a.kbps, a.nkb - t.kb0);
    return t;
  };

  if (warp == S::kEpiWarps) {
    // ------------------------------------------------ loads (one thread)
    if (lane == 0) {
      uint32_t it = 0;  // K-blocks so far
      bool ok = true;
      const uint32_t full0 = CG == 2 ? mapa(smem_u32(&bars->full[0]), 0) : smem_u32(&bars->full[0]);
      for (int u = unit0; u < units && ok; u += units_step) {
        const Unit t = unit_of(u);
        for (int sg = 0; sg < a.nseg && ok; ++sg) {
          const int za = a.pa[sg] + t.batch, zb = a.pb[sg];
          for (int k = 0; k < t.kbn; ++k, ++it) {
            const int st = int(it % STAGES);
            if (it >= STAGES && !(ok = mbar_wait(&bars->empty[st], ((it / STAGES) - 1) & 1u))) break;
            const uint32_t bar = full0 + uint32_t(st) * 8u;
            if (rank == 0) mbar_arrive_expect_tx(&bars->full[st], uint32_t(CG * S::STAGE));
            const uint32_t sa = smem_u32(sm + st * S::STAGE), sb = sa + S::A_BYTES;
            const int kx = (t.kb0 + k) * kBK;
            if (AMN) {
              tma_load_3d<CG>(sa, &mapA, t.m0, kx, za, bar);
              tma_load_3d<CG>(sa + 8192, &mapA, t.m0 + 64, kx, za, bar);
            } else {
              tma_load_3d<CG>(sa, &mapA, kx, t.m0, za, bar);
            }
            if (GATED) {
              if (CG == 2) {  // the gate half in one CTA, the up half in the other
                tma_load_3d<CG>(sb, &mapB, kx, t.n0, 2 * zb + int(rank), bar);
              } else {
                tma_load_3d<CG>(sb, &mapB, kx, t.n0, 2 * zb, bar);
                tma_load_3d<CG>(sb + S::B_BYTES / 2, &mapB, kx, t.n0, 2 * zb + 1, bar);
              }
            } else if (BMN) {
#pragma unroll
              for (int j = 0; j < S::BNC / 64; ++j)
                tma_load_3d<CG>(sb + j * 8192, &mapB, t.n0 + int(rank) * S::BNC + 64 * j, kx, zb, bar);
            } else {
              tma_load_3d<CG>(sb, &mapB, kx, t.n0 + int(rank) * S::BNC, zb, bar);
            }
          }
        }
      }
      // the last loads have landed before the CTA may end (bounded)
      if (!ok) atomicExch(&bars->abort_, 1);
      for (uint32_t j = it > uint32_t(STAGES) ? it - STAGES : 0; rank == 0 && j < it; ++j)
        if (!mbar_wait(&bars->full[j % STAGES], (j / STAGES) & 1u)) atomicExch(&bars->abort_, 1);
    }
    __syncwarp();
  } else if (warp == S::kEpiWarps + 1) {
    // ------------------------------------------------ MMAs (one thread of the cluster)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t ID = (1u << 4) | (KIND == kBf16 ? (1u << 7) | (1u << 10) : 0u) | (AMN ? 1u << 15 : 0u) |
                              (BMN ? 1u << 16 : 0u) | (uint32_t(BN >> 3) << 17) | (uint32_t((128 * CG) >> 4) << 24);
      uint32_t it = 0, run = 0;
      bool ok = true;
      for (int u = unit0; u < units && ok; u += units_step) {
        const Unit t = unit_of(u);
        int left = a.nseg * t.kbn, len = left;
        if (PROMOTE) len = a.nseg > a.nbig ? (a.nseg - a.nbig) * t.kbn : min(left, kRun);
        for (; left > 0 && ok; ++run) {
          const uint32_t acc = run & 1u;
          if (run >= 2 && !(ok = mbar_wait(&bars->tempty[acc], ((run >> 1) - 1) & 1u))) break;
          tc_fence_after();
          const uint32_t d = tbase + acc * BN;
          for (int k = 0; k < len; ++k, ++it) {
            const uint32_t st = it % STAGES;
            if (!(ok = mbar_wait(&bars->full[st], (it / STAGES) & 1u))) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(sm + st * S::STAGE), sb = sa + S::A_BYTES;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma<CG, KIND>(d, AMN ? mn_desc(sa + kk * 2048) : sw128_kmajor_desc(sa + kk * 32),
                            BMN ? mn_desc(sb + kk * 2048) : sw128_kmajor_desc(sb + kk * 32), ID, (k | kk) ? 1u : 0u);
            mma_commit<CG>(&bars->empty[st]);
          }
          if (ok) mma_commit<CG>(&bars->tfull[acc]);
          left -= len;
          len = min(left, kRun);
        }
      }
      if (!ok) atomicExch(&bars->abort_, 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue
    const int q = warp & 3, grp = warp >> 2;
    uint8_t* buf0 = sE + warp * (NBUF * 4096);
    const uint32_t lane_base = uint32_t(q * 32) << 16;
    constexpr bool IN = (EPI == kEpiFwd && !GATED) || EPI == kEpiDz;
    constexpr int RING = IN && EPI == kEpiDz && GATED ? 2 : NBUF;  // (a gated dz: the third buffer holds du)
    constexpr int AHEAD = RING - 1;                                // input items in flight
    const bool has_in = IN && (EPI == kEpiDz || a.has_in);
    const TO* in = static_cast<const TO*>(a.in);
    TO* out = static_cast<TO*>(a.out);
    constexpr int halves = GATED ? 2 : 1;
    // columns this item kind walks: accumulator columns for partial sums of a gated layer
    constexpr int WALK = GATED && EPI == kEpiPart ? BN : ON;
    constexpr int NCH = WALK / CW;
    const uint32_t tempty0 = CG == 2 ? mapa(smem_u32(&bars->tempty[0]), 0) : smem_u32(&bars->tempty[0]);
    const bool vec_b = a.bias && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
    const bool vec_bu = vec_b && a.N % 4 == 0;
    const bool vec_s = a.ws && (reinterpret_cast<uintptr_t>(a.ws) & 15) == 0;
    const bool vec_su = vec_s && a.N % 4 == 0;

    // the input of the warp's items, in order: (unit, chunk) pairs with a row and a column inside
    int pu = unit0, pc = grp;
    uint32_t pi = 0;  // items whose input was asked for
    auto prefetch = [&]() {  // lane 0, TMA inputs
      while (pu < units) {
        const Unit t = unit_of(pu);
        const int row = t.m0 + 32 * q, col = t.n0 + pc * CW;
        const bool good = row < a.M && col < a.N;
        const int c = pc;
        pc += 2;
        if (pc >= NCH) pc = grp, pu += units_step;
        if (good && c < NCH) {
          uint64_t* bar = &bars->in[warp][pi % RING];
          mbar_arrive_expect_tx(bar, 4096);
          tma_load_3d<1>(smem_u32(buf0 + (pi % RING) * 4096), &mapI, col, row, 0, smem_u32(bar));
          ++pi;
          return;
        }
      }
    };
    if (has_in && a.in_tma && lane == 0)
      for (int i = 0; i < AHEAD; ++i) prefetch();

    uint32_t item = 0, run = 0;
    bool ok = true;
    constexpr bool PAIR = GATED && EPI != kEpiPart;  // an item takes gate and up accumulators
    constexpr int NI = (NCH + 1) / 2;                // items per warp and tile
    auto wait_run = [&]() {                          // the run's accumulator is complete
      if (*aborted) ok = false;
      if (ok && lane == 0) ok = mbar_wait(&bars->tfull[run & 1u], (run >> 1) & 1u);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after();
      return ok;
    };
    auto done_run = [&]() {  // and may be overwritten
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + (run & 1u) * 8u);
      ++run;
    };
    for (int u = unit0; u < units && ok; u += units_step) {
      const Unit t = unit_of(u);
      const int row0 = t.m0 + 32 * q, row = row0 + lane;
      const bool live = row < a.M;
      // one item: 32 rows by CW columns. PROMOTE: pg, pu_ hold its sums
      auto do_item = [&](int c, uint32_t tacc, float* pg, float* pu_) {
        const int col0 = WALK == BN && GATED ? t.n0 + (c * CW) % ON : t.n0 + c * CW;
        if (row0 >= a.M || col0 >= a.N) return;
        uint8_t* buf = buf0 + (item % RING) * 4096;
        if (has_in) {
          if (a.in_tma) {
            if (lane == 0) ok = mbar_wait(&bars->in[warp][item % RING], (item / RING) & 1u);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) return;
          } else {  // rows side by side across the lanes
            constexpr int RB = 16;  // rows in flight
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += RB) {
              TO v[RB][CW / 32];
#pragma unroll
              for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int j = 0; j < CW / 32; ++j) {
                  const int e = lane + 32 * j;
                  v[r][j] = TO(0.f);
                  if (row0 + r0 + r < a.M && col0 + e < a.N) v[r][j] = in[(long long)(row0 + r0 + r) * a.ldi + col0 + e];
                }
#pragma unroll
              for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int j = 0; j < CW / 32; ++j) {
                  const int byte = (lane + 32 * j) * int(sizeof(TO));
                  *reinterpret_cast<TO*>(buf + (r0 + r) * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15)) = v[r][j];
                }
            }
            __syncwarp();
          }
        }
        if (EPI == kEpiDz && GATED) {  // du's buffer is free once the last item's stores have read it
          if (lane == 0) {
            bulk_wait_read<0>();
            if (a.in_tma) {
              fence_proxy_async_smem();
              prefetch();
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < CW / 32; ++h) {  // 32 columns at a time
          const int col = col0 + 32 * h;
          float g_[32], up_[PAIR ? 32 : 1];
          float* g = g_;
          float* up = up_;
          if (PROMOTE) {  // (CW = 32: one pass)
            g = pg;
            up = pu_;
          } else {
            const uint32_t tc = tacc + uint32_t(c * CW + 32 * h);
            tmem_ld32(tc, g);
            if (PAIR) tmem_ld32(tc + ON, up);
            tmem_ld_wait();
          }
          if (EPI == kEpiFwd || EPI == kEpiDz) {
            if (KIND == kE4m3) {
              const float xs = live ? __ldg(a.xs + row) : 0.f;
              float w[32];
              load_cols(a.ws, col, a.N, vec_s, w);
#pragma unroll
              for (int k = 0; k < 32; ++k) g[k] *= xs * w[k];
              if (GATED) {
                load_cols(a.ws + a.N, col, a.N, vec_su, w);
#pragma unroll
                for (int k = 0; k < 32; ++k) up[GATED ? k : 0] *= xs * w[k];
              }
            }
            if (a.bias) {
              float b[32];
              load_cols(a.bias, col, a.N, vec_b, b);
#pragma unroll
              for (int k = 0; k < 32; ++k) g[k] += b[k];
              if (GATED) {
                load_cols(a.bias + a.N, col, a.N, vec_bu, b);
#pragma unroll
                for (int k = 0; k < 32; ++k) up[GATED ? k : 0] += b[k];
              }
            }
          }
          float x[IN ? 32 : 1];  // the input's 32 columns of this row
          if (has_in) {
#pragma unroll
            for (int k = 0; k < int(sizeof(TO)) * 2; ++k) {
              const int slot = h * 4 + k;
              const uint4 v = *reinterpret_cast<const uint4*>(buf + lane * 128 + ((slot ^ (lane & 7)) << 4));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (sizeof(TO) == 4) {
                  x[IN ? 4 * k + e : 0] = __uint_as_float(w[e]);
                } else {
                  x[IN ? (8 * k + 2 * e) & 31 : 0] = __uint_as_float(w[e] << 16);
                  x[IN ? (8 * k + 2 * e + 1) & 31 : 0] = __uint_as_float(w[e] & 0xffff0000u);
                }
              }
            }
          }
          if (EPI == kEpiFwd) {
            switch (a.act) {
              case DSF_ACT_RELU: act_fwd<DSF_ACT_RELU, GATED>(g, up); break;
              case DSF_ACT_SILU: act_fwd<DSF_ACT_SILU, GATED>(g, up); break;
              case DSF_ACT_GELU: act_fwd<DSF_ACT_GELU, GATED>(g, up); break;
              default: act_fwd<DSF_ACT_NONE, GATED>(g, up);
            }
            if (has_in) {
#pragma unroll
              for (int k = 0; k < 32; ++k) g[k] += x[IN ? k : 0];
            }
          }
          if (EPI == kEpiDz) {
            switch (a.act) {
              case DSF_ACT_RELU: act_bwd<DSF_ACT_RELU, GATED>(x, g, up); break;
              case DSF_ACT_SILU: act_bwd<DSF_ACT_SILU, GATED>(x, g, up); break;
              case DSF_ACT_GELU: act_bwd<DSF_ACT_GELU, GATED>(x, g, up); break;
              default: act_bwd<DSF_ACT_NONE, GATED>(x, g, up);
            }
          }
          auto put = [&](uint8_t* b, const float* v) {
#pragma unroll
            for (int k = 0; k < int(sizeof(TO)) * 2; ++k) {
              const int slot = h * 4 + k;
              uint4 w;
              if (sizeof(TO) == 4)
                w = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                               __float_as_uint(v[4 * k + 3]));
              else
                w = make_uint4(pack_bf16x2(v[(8 * k) & 31], v[(8 * k + 1) & 31]),
                               pack_bf16x2(v[(8 * k + 2) & 31], v[(8 * k + 3) & 31]),
                               pack_bf16x2(v[(8 * k + 4) & 31], v[(8 * k + 5) & 31]),
                               pack_bf16x2(v[(8 * k + 6) & 31], v[(8 * k + 7) & 31]));
              *reinterpret_cast<uint4*>(b + lane * 128 + ((slot ^ (lane & 7)) << 4)) = w;
            }
          };
          put(buf, g);
          if (EPI == kEpiDz && GATED) put(buf0 + 2 * 4096, up);
          if (EPI == kEpiDz && a.part) {
            const float s = column_sum(g, lane);
            float* p = a.part + (long long)(row0 >> 5) * (halves * a.N);
            if (col + lane < a.N) p[col + lane] = s;
            if (GATED) {
              const float s2 = column_sum(up, lane);
              if (col + lane < a.N) p[a.N + col + lane] = s2;
            }
          }
        }
        // the item's output
        int plane = t.batch;
        if (EPI == kEpiPart) plane = GATED ? t.split * 2 + (c * CW) / ON : t.split * a.nb + t.batch;
        fence_proxy_async_smem();
        __syncwarp();
        if (a.out_tma) {
          if (lane == 0) {
            tma_store_3d(&mapO, col0, row0, plane, smem_u32(buf));
            if (EPI == kEpiDz && GATED) tma_store_3d(&mapO, col0, row0, 1, smem_u32(buf0 + 2 * 4096));
            bulk_commit();
          }
        } else {
          TO* o = out + plane * a.out_plane;
#pragma unroll 8
          for (int r = 0; r < 32; ++r)
#pragma unroll
            for (int j = 0; j < CW / 32; ++j) {
              const int e = lane + 32 * j, byte = e * int(sizeof(TO));
              const int at = r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
              if (row0 + r < a.M && col0 + e < a.N)
                o[(long long)(row0 + r) * a.ldo + col0 + e] = *reinterpret_cast<const TO*>(buf + at);
            }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!(EPI == kEpiDz && GATED)) {
          // the buffer that the next item (or its input's load) takes is free
          if (lane == 0) {
            bulk_wait_read<1>();
            if (has_in && a.in_tma) prefetch();
          }
          __syncwarp();
        }
        ++item;
      };
      if (PROMOTE) {
        float sum[NI][PAIR ? 2 : 1][32];
        const int runs = runs_of<PROMOTE>(a, t.kbn);
        for (int r = 0; r < runs; ++r) {
          if (!wait_run()) break;
          const uint32_t tacc = tbase + (run & 1u) * BN + lane_base;
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
              float v[32];
              tmem_ld32(tacc + uint32_t((grp + 2 * i) * CW + h * ON) % BN, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) sum[i][h][k] = r ? sum[i][h][k] + v[k] : v[k];
            }
          done_run();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (ok && grp + 2 * i < NCH) do_item(grp + 2 * i, 0, sum[i][0], sum[i][PAIR ? 1 : 0]);
      } else {
        if (!wait_run()) break;
        const uint32_t tacc = tbase + (run & 1u) * BN + lane_base;
#pragma unroll 1
        for (int c = grp; c < NCH && ok; c += 2) do_item(c, tacc, nullptr, nullptr);
        if (!ok) break;
        done_run();
      }
    }
    if (!ok && lane == 0) atomicExch(&bars->abort_, 1);
    if (lane == 0) {
      // (an aborted run: inputs asked for and not taken)
      for (uint32_t i = item; has_in && a.in_tma && i < pi; ++i) mbar_wait(&bars->in[warp][i % RING], (i / RING) & 1u);
      bulk_wait_all();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    tmem_dealloc_cg<CG>(tbase, S::TCOLS);
  }
  if (threadIdx.x == 0 && bars->abort_ && a.status) atomicOr(a.status, DSF_FLAG_TIMEOUT);
}

// ---------------------------------------------------------------- host side
// A matrix of the products, as [planes][rows][cols] elements.
struct Mat {
  const void* p;
  long long rows, cols, ld, planes, plane;  // ld, plane: strides in elements
};

// One product; fills in tiles and splits' bookkeeping and launches. false:
// a launch or a tensor map failed.
struct Product {
  TcArgs a;
  Mat A, B, in, out;
  int major;
  bool gated, f32;  // f32: fp32 operands (in terms) and outputs
  int epi, cfg;  // cfg: 0: CG 2, 1: CG 1 x BN 128, 2: CG 1 x BN 64
};

bool tensor_map_3d(CUtensorMap* m, const Mat& x, int esize, bool f32, int box_cols, int box_rows);
bool run_fwd_product(const Product& p, cudaStream_t s);   // K-major, bf16 operands
bool run_e4m3_product(const Product& p, cudaStream_t s);  // K-major, e4m3 operands
bool run_dz_product(const Product& p, cudaStream_t s);
bool run_grad_product(const Product& p, cudaStream_t s);  // MN-major operands

template <int CG, int BN, int MAJOR, int KIND, bool GATED, int EPI, class TO, bool PROMOTE>
bool launch_tc(const Product& p, cudaStream_t s) {
  using S = Shape<CG, BN, GATED, EPI>;
  auto* kernel = tc_kernel<CG, BN, MAJOR, KIND, GATED, EPI, TO, PROMOTE>;
  static int grid_max[64] = {};  // (host threads may race on it: each computes the same value)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 1 : 0;
  if (grid_max[dev] == 0) {
    int sms = 0, n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return false;
    if (CG == 2) {
      cfg.gridDim = dim3(unsigned(sms / 2 * 2));
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return false;
      grid_max[dev] = 2 * n;
    } else {
      grid_max[dev] = sms;
    }
  }
  const long long units = (long long)p.a.mt * p.a.nt * p.a.nb * p.a.splits;
  if (units <= 0 || units * CG > INT32_MAX) return false;
  const long long g = units * CG < grid_max[dev] ? units * CG : grid_max[dev];
  cfg.gridDim = dim3(unsigned(g));
  constexpr int es = KIND == kBf16 ? 2 : 1;
  CUtensorMap mA, mB, mI, mO;
  if (!tensor_map_3d(&mA, p.A, es, false, MAJOR == kNN ? 64 : 128 / es, MAJOR == kNN ? 64 : 128)) return false;
  if (!tensor_map_3d(&mB, p.B, es, false, MAJOR != kKK ? 64 : 128 / es,
                     MAJOR != kKK ? 64 : (GATED && CG == 1 ? BN / 2 : BN / CG)))
    return false;
  constexpr int cw = 128 / int(sizeof(TO));
  mI = mA;
  mO = mA;
  if (p.a.has_in && p.a.in_tma && !tensor_map_3d(&mI, p.in, sizeof(TO), sizeof(TO) == 4, cw, 32)) return false;
  if (p.a.out_tma && !tensor_map_3d(&mO, p.out, sizeof(TO), sizeof(TO) == 4, cw, 32)) return false;
  return cudaLaunchKernelEx(&cfg, kernel, p.a, mA, mB, mI, mO) == cudaSuccess;
}

// Tile configurations: accumulator columns (an fp32 product's wide tiles are
// half as wide) and rows.
constexpr int cfg_bn(int cfg, bool promote) { return cfg == 0 ? (promote ? 128 : 256) : (cfg == 1 ? 128 : 64); }
constexpr int cfg_rows(int cfg) { return cfg == 0 ? 256 : 128; }

template <int MAJOR, int KIND, bool GATED, int EPI, class TO, bool PROMOTE>
bool launch_cfg(const Product& p, cudaStream_t s) {
  if (p.cfg == 0) return launch_tc<2, cfg_bn(0, PROMOTE), MAJOR, KIND, GATED, EPI, TO, PROMOTE>(p, s);
  if (p.cfg == 1) return launch_tc<1, 128, MAJOR, KIND, GATED, EPI, TO, PROMOTE>(p, s);
  if constexpr (!GATED) return launch_tc<1, 64, MAJOR, KIND, GATED, EPI, TO, PROMOTE>(p, s);
  return false;
}

}  // namespace dense
}  // namespace dsf
