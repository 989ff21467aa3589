// The matrix products of the dense operators on the tensor cores: D = A B^T
// with the operator's epilogue, sums in fp32.
//
// One persistent, warp-specialised kernel. A work unit is a tile of 128 CG x
// BN accumulators (CG CTAs of a cluster work on one tile together: CG = 2
// halves what each SM has to read of B), over all of K or one K-split.
//   warp 16  brings A and B by TMA: K-blocks of 128 bytes per row in the
//            128-byte swizzle, through a ring of stages;
//   warp 17  issues the MMAs (tcgen05.mma, in the cluster's first CTA) into
//            one of two accumulators in tensor memory;
//   warps 0-15 run the epilogue of the other accumulator, in items of 32 rows
//            (a warp's lane quarter, one row per lane) by 32 columns. Inputs
//            (the residual, or the upstream gradient; loaded an item ahead)
//            and outputs change between a row per lane and 16 bytes of
//            neighbouring lanes in a 2 or 4 KB buffer per warp, so that
//            global memory sees whole row segments. (Not by TMA: its stores
//            and loads queue behind the operands' loads, 2 us an item.)
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
#include <type_traits>

#include "dense_math.cuh"
#include "dinsparse.h"
#include "pdl.cuh"
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

// Division of unsigned 32-bit numbers by a fixed divisor: q = (mulhi(n, m) + n) >> l
// with l = ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1, exact for every n below 2^31.
struct Div {
  uint32_t d, m, l;
};
inline Div make_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return Div{d, uint32_t(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const Div& v) { return (__umulhi(n, v.m) + n) >> v.l; }

struct TcArgs {
  int M, N;          // rows; output columns (a gated layer's: F)
  int mt, nt, nb;    // tiles along M and N, batches (halves of dW)
  Div by_splits, by_batch, by_group, by_last;  // splits; mt nt; 8 nt; M tiles of the last group of 8
  int nkb, kbps;     // K-blocks per segment, per split
  int nbig;          // PROMOTE: the last nbig segments are the products of leading terms
  int splits, nseg;
  uint8_t pa[kMaxSeg], pb[kMaxSeg];  // the segments' planes (A: + batch; B of a gated layer: 2 pb, 2 pb + 1)
  int act;
  const float *bias, *xs, *ws;  // z = acc * xs[m] * ws[n] + bias[n] (each nullable; the up half at n + N)
  const void* in;            // nullable unless kEpiDz
  long long ldi;
  void* out;
  long long ldo, out_plane;  // strides in elements
  int in_vec, out_vec;       // rows at 16-byte boundaries
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
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
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
// An arrival that orders nothing but itself: what it announces (accumulators
// read, tcgen05.wait::ld done) is complete in registers. A release would wait
// for the thread's global stores.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
template <int CG, int BN, bool GATED, int EPI, class TO>
struct Shape {
#ifndef DZW
#define DZW 8
#endif
  static constexpr int kEpiWarps = GATED && sizeof(TO) == 4 && EPI != kEpiPart ? 8 : (GATED && EPI == kEpiDz ? DZW : 16), kThreads = 32 * (kEpiWarps + 2);
  static constexpr int kGroups = kEpiWarps / 4;  // warps on one lane quarter
  static constexpr int ITEM = 32 * 32 * int(sizeof(TO));
  static constexpr int BNC = BN / CG;            // B rows (or MN-major columns) in this CTA
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BNC * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int EBYTES = kEpiWarps * ITEM;
  static constexpr int kRoom = 227 * 1024 - 1024 - 256 - EBYTES;
  static constexpr int STAGES = kRoom / STAGE < 8 ? kRoom / STAGE : 8;
  static constexpr int SMEM = STAGES * STAGE + EBYTES + 256 + 1024;
  static constexpr uint32_t TCOLS = 2 * BN;      // two accumulators
  static_assert(TCOLS <= 512 && (TCOLS & (TCOLS - 1)) == 0, "tensor memory columns");
  static_assert(STAGES >= 3, "ring");
  static_assert(B_BYTES % (GATED && CG == 1 ? 2048 : 1024) == 0, "swizzle atoms");
};

struct Bars {
  uint64_t full[8], empty[8], tfull[2], tempty[2];
  uint32_t tmem;
  int abort_;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

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

// ---------------------------------------------------------------- the kernel
constexpr int kRun = 4;  // PROMOTE: K-blocks of leading terms per run

// Accumulator runs of a unit with kbn K-blocks per segment.
template <bool PROMOTE>
__device__ __forceinline__ int runs_of(const TcArgs& a, int kbn) {
  return PROMOTE ? (a.nseg > a.nbig ? 1 : 0) + (a.nbig * kbn + kRun - 1) / kRun : 1;
}

template <int CG, int BN, int MAJOR, int KIND, bool GATED, int EPI, class TO, bool PROMOTE>
__global__ void __launch_bounds__(Shape<CG, BN, GATED, EPI, TO>::kThreads, 1)
    tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap mapA,
              const __grid_constant__ CUtensorMap mapB) {
  using S = Shape<CG, BN, GATED, EPI, TO>;
  constexpr bool AMN = MAJOR == kNN, BMN = MAJOR != kKK;
  constexpr int kBK = KIND == kBf16 ? 64 : 128;            // K elements per block (128 bytes)
  constexpr int ON = GATED ? BN / 2 : BN;                  // output columns per tile
  constexpr int CW = 32;                                   // output columns per item
  constexpr int ROWB = CW * int(sizeof(TO));               // an item row's bytes
  constexpr int STAGES = S::STAGES;
  static_assert(!(GATED && BMN), "a gated layer's product is K-major");
  extern __shared__ uint8_t dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* sE = sm + STAGES * S::STAGE;
  Bars* bars = reinterpret_cast<Bars*>(sE + S::EBYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int unit0 = blockIdx.x / CG, units_step = gridDim.x / CG;
  const int tiles = a.mt * a.nt * a.nb, units = tiles * a.splits;

  if (warp == S::kEpiWarps && lane == 0) {
    prefetch_map(&mapA);
    prefetch_map(&mapB);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->tfull[i], 1);
      mbar_init(&bars->tempty[i], S::kEpiWarps * CG);
    }
    bars->abort_ = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  pdl_go();
  // (the loads start while tensor memory is being allocated)
  uint32_t tbase = 0;
  if (warp != S::kEpiWarps) {
    if (warp == S::kEpiWarps + 1) {
      tmem_alloc_cg<CG>(&bars->tmem, S::TCOLS);
      tmem_relinquish_cg<CG>();
      tc_fence_before();
    }
    asm volatile("bar.sync 1, %0;" ::"n"(S::kThreads - 32) : "memory");
    tc_fence_after();
    tbase = bars->tmem;
  }
  volatile int* aborted = &bars->abort_;

  // a unit: split-minor, then N tiles within groups of M tiles, so that the
  // units in flight share rows of A and of B in L2
  struct Unit {
    int m0, n0, batch, split, kb0, kbn;
  };
  auto unit_of = [&](int u) {
    Unit t;
    uint32_t r = div_by(u, a.by_splits);
    t.split = u - int(r) * a.splits;
    t.batch = int(div_by(r, a.by_batch));
    r -= uint32_t(t.batch) * a.by_batch.d;
    const uint32_t grp = div_by(r, a.by_group);
    r -= grp * a.by_group.d;
    const bool whole = int(grp * 8 + 8) <= a.mt;
    const uint32_t n = whole ? r >> 3 : div_by(r, a.by_last), gm = whole ? 8 : a.by_last.d;
    t.m0 = int(grp * 8 + r - n * gm) * 128 * CG + int(rank) * 128;
    t.n0 = int(n) * ON;
    t.kb0 = t.split * a.kbps;
    t.kbn = min(a.kbps, a.nkb - t.kb0);
    return t;
  };

  if (warp == S::kEpiWarps) {
    // ------------------------------------------------ loads (one thread)
    if (lane == 0) {
      pdl_wait();
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
    pdl_wait();
    const int q = warp & 3, grp = warp >> 2;
    uint8_t* buf = sE + warp * S::ITEM;
    const uint32_t lane_base = uint32_t(q * 32) << 16;
    constexpr bool IN = (EPI == kEpiFwd && !GATED) || EPI == kEpiDz;
    constexpr int GR = S::kGroups;
    // byte `at` of an item's row r; 16-byte slots XOR-swizzled by the row, so that neither a
    // slot of 8 rows nor whole rows meet in a bank
    auto slot = [](int r, int at) {
      return r * ROWB + (((at >> 4) ^ (ROWB == 64 ? (r >> 1) & 3 : r & 7)) << 4) + (at & 15);
    };
    const bool has_in = IN && (EPI == kEpiDz || a.in);
    const TO* in = static_cast<const TO*>(a.in);
    TO* out = static_cast<TO*>(a.out);
    constexpr int halves = GATED ? 2 : 1;
    // columns this item kind walks: accumulator columns for partial sums of a gated layer
    constexpr int WALK = GATED && EPI == kEpiPart ? BN : ON;
    constexpr int NCH = WALK / CW;
    const uint32_t tempty0 = CG == 2 ? mapa(smem_u32(&bars->tempty[0]), 0) : smem_u32(&bars->tempty[0]);
    constexpr bool COLS = EPI == kEpiFwd || EPI == kEpiDz, SCALED = KIND == kE4m3 && EPI == kEpiFwd;
    // columns j .. j + 7 of this lane's row, from and to an item's buffer
    auto get8 = [&](const uint8_t* b, int j, float* v) {
#pragma unroll
      for (int k = 0; k < int(sizeof(TO)) / 2; ++k) {
        const uint4 u = *reinterpret_cast<const uint4*>(b + slot(lane, j * int(sizeof(TO)) + 16 * k));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (sizeof(TO) == 4) {
            v[4 * k + e] = __uint_as_float(w[e]);
          } else {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
          }
        }
      }
    };
    auto put8 = [&](uint8_t* b, int j, const float* v) {
#pragma unroll
      for (int k = 0; k < int(sizeof(TO)) / 2; ++k) {
        uint4 w;
        if (sizeof(TO) == 4)
          w = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                         __float_as_uint(v[4 * k + 3]));
        else
          w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        *reinterpret_cast<uint4*>(b + slot(lane, j * int(sizeof(TO)) + 16 * k)) = w;
      }
    };

    // A 16-byte piece of an item for each lane: 4 (bf16) or 8 (fp32) lanes side
    // by side on a row. Pieces past the matrix's edge element by element.
    constexpr int EL = 16 / int(sizeof(TO)), LPR = CW / EL, RPI = 32 / LPR, NV = 32 / RPI;
    const int piece_row = lane / LPR, piece_col = lane % LPR * EL;
    auto load_item = [&](uint4* v, int r0, int c0) {
      const int cc = c0 + piece_col;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = r0 + i * RPI + piece_row;
        const TO* p = in + (long long)r * a.ldi + cc;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r >= a.M || cc >= a.N) continue;
        if (cc + EL <= a.N) {
          v[i] = __ldg(reinterpret_cast<const uint4*>(p));
        } else {
          uint32_t w[4] = {};
#pragma unroll
          for (int e = 0; e < EL - 1; ++e)
            if (cc + e < a.N) {
              if (sizeof(TO) == 4) w[e] = __float_as_uint(to_float(p[e]));
              else w[e / 2] |= (__float_as_uint(to_float(p[e])) >> 16) << (16 * (e & 1));
            }
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    auto store_item = [&](TO* base, int r0, int c0) {  // from the buffer
      __syncwarp();
      if (a.out_vec) {
        const int cc = c0 + piece_col;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int rr = i * RPI + piece_row, r = r0 + rr;
          const uint8_t* b = buf + slot(rr, piece_col * int(sizeof(TO)));
          TO* p = base + (long long)r * a.ldo + cc;
          if (r >= a.M || cc >= a.N) continue;
          if (cc + EL <= a.N) {
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(b);
          } else {
            for (int e = 0; cc + e < a.N; ++e) p[e] = reinterpret_cast<const TO*>(b)[e];
          }
        }
      } else {
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
          if (r0 + r < a.M && c0 + lane < a.N)
            base[(long long)(r0 + r) * a.ldo + c0 + lane] =
                *reinterpret_cast<const TO*>(buf + slot(r, lane * int(sizeof(TO))));
      }
      __syncwarp();
    };
    // The input of the warp's next item ((unit, item) pairs in order), where it
    // can be loaded in pieces: bf16 into registers; fp32, whose sums take the
    // registers, as far as L2.
    constexpr bool PRE = IN && sizeof(TO) == 2;
    uint4 pin[PRE ? NV : 1];
    auto prefetch = [&](int u, int c) {
      if (!IN) return;
      if (c >= NCH) c = grp, u += units_step;
      const bool any = has_in && a.in_vec && u < units && c < NCH;
      const Unit t = unit_of(any ? u : unit0);
      if (PRE) {
        load_item(pin, any ? t.m0 + 32 * q : a.M, t.n0 + c * CW);
      } else if (any) {
        const int r = t.m0 + 32 * q + lane, cc = t.n0 + c * CW;
        if (r < a.M && cc < a.N) prefetch_l2(in + (long long)r * a.ldi + cc);
      }
    };
    prefetch(unit0, grp);
    // bias and scales of an item's columns, one column per lane: handed round by
    // shuffles (the L1 that 220 KB of shared memory leave does not keep them)
    struct Cols {
      float b, bu, s, su;
    };
    auto load_cols = [&](int c0) {
      Cols v = {0.f, 0.f, 1.f, 1.f};
      if (COLS && c0 + lane < a.N) {
        const int n = c0 + lane;
        if (a.bias) {
          v.b = __ldg(a.bias + n);
          if (GATED) v.bu = __ldg(a.bias + a.N + n);
        }
        if (SCALED) {
          v.s = __ldg(a.ws + n);
          if (GATED) v.su = __ldg(a.ws + a.N + n);
        }
      }
      return v;
    };

    uint32_t run = 0;
    bool ok = true;
    constexpr bool PAIR = GATED && EPI != kEpiPart;  // an item takes gate and up accumulators
    constexpr int NI = (NCH + GR - 1) / GR;          // items per warp and tile
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
        if (row0 >= a.M || col0 >= a.N) {
          prefetch(u, c + GR);
          return;
        }
        if (has_in) {
          if (a.in_vec) {
            if (!PRE) {
              uint4 v[NV];
              load_item(v, row0, col0);
#pragma unroll
              for (int i = 0; i < NV; ++i)
                *reinterpret_cast<uint4*>(buf + slot(i * RPI + piece_row, piece_col * int(sizeof(TO)))) = v[i];
            } else {
#pragma unroll
              for (int i = 0; i < NV; ++i)
                *reinterpret_cast<uint4*>(buf + slot(i * RPI + piece_row, piece_col * int(sizeof(TO)))) = pin[PRE ? i : 0];
            }
          } else {  // one column per lane, 16 rows in flight
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 16) {
              TO v[16];
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                v[r] = TO(0.f);
                if (row0 + r0 + r < a.M && col0 + lane < a.N) v[r] = in[(long long)(row0 + r0 + r) * a.ldi + col0 + lane];
              }
#pragma unroll
              for (int r = 0; r < 16; ++r)
                *reinterpret_cast<TO*>(buf + slot(r0 + r, lane * int(sizeof(TO)))) = v[r];
            }
          }
          __syncwarp();
        }
        const Cols cols = load_cols(col0);
        const float xs = SCALED && live ? __ldg(a.xs + row) : 0.f;
        // g (and up): the accumulators of this lane's row, then the outputs
        float g_[32], up_[PAIR ? 32 : 1];
        float* g = g_;
        float* up = up_;
        if (PROMOTE) {
          g = pg;
          up = pu_;
        } else {
          tmem_ld32(tacc + uint32_t(c * CW), g);
          if (PAIR) tmem_ld32(tacc + uint32_t(c * CW) + ON, up);
          tmem_ld_wait();
        }
        // eight columns at a time, from the accumulators to the item's buffers
        auto math = [&](auto act_tag) {
          constexpr int ACT = decltype(act_tag)::value;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float* v = g + j;
            float* w = up + (PAIR ? j : 0);
            if (COLS) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float b = __shfl_sync(0xffffffffu, cols.b, j + k);
                v[k] = SCALED ? fmaf(v[k], xs * __shfl_sync(0xffffffffu, cols.s, j + k), b) : v[k] + b;
                if (PAIR) {
                  const float bu = __shfl_sync(0xffffffffu, cols.bu, j + k);
                  w[PAIR ? k : 0] = SCALED ? fmaf(w[PAIR ? k : 0], xs * __shfl_sync(0xffffffffu, cols.su, j + k), bu)
                                           : w[PAIR ? k : 0] + bu;
                }
              }
            }
            float x[8];
            if (has_in) get8(buf, j, x);
            if (EPI == kEpiFwd) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[k] = act_value<ACT>(v[k]);
                if (PAIR) v[k] *= w[PAIR ? k : 0];
                if (has_in) v[k] += x[k];
              }
            }
            if (EPI == kEpiDz) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float2 f = act_both<ACT>(v[k]);
                v[k] = (PAIR ? x[k] * w[PAIR ? k : 0] : x[k]) * f.y;
                if (PAIR) w[PAIR ? k : 0] = x[k] * f.x;
              }
            }
            put8(buf, j, v);
          }
        };
        if (EPI == kEpiFwd || EPI == kEpiDz) {
          switch (a.act) {
            case DSF_ACT_RELU: math(std::integral_constant<int, DSF_ACT_RELU>{}); break;
            case DSF_ACT_SILU: math(std::integral_constant<int, DSF_ACT_SILU>{}); break;
            case DSF_ACT_GELU: math(std::integral_constant<int, DSF_ACT_GELU>{}); break;
            default: math(std::integral_constant<int, DSF_ACT_NONE>{});
          }
        } else {
          math(std::integral_constant<int, DSF_ACT_NONE>{});
        }
        // (a gated dz: du takes the buffer after dg has left it)
        int plane = t.batch;
        if (EPI == kEpiPart) plane = GATED ? t.split * 2 + (c * CW) / ON : t.split * a.nb + t.batch;
        store_item(out + plane * a.out_plane, row0, col0);
        if (EPI == kEpiDz && PAIR) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) put8(buf, j, up + (PAIR ? j : 0));
          store_item(out + a.out_plane, row0, col0);
        }
        if (EPI == kEpiDz && a.part) {
          float* p = a.part + (long long)(row0 >> 5) * (halves * a.N) + col0 + lane;
          const float s = column_sum(g, lane);
          if (col0 + lane < a.N) p[0] = s;
          if (PAIR) {
            const float s2 = column_sum(up, lane);
            if (col0 + lane < a.N) p[a.N] = s2;
          }
        }
        prefetch(u, c + GR);
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
              if (grp + GR * i >= NCH) continue;
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                float v[16];
                tmem_ld16(tacc + uint32_t((grp + GR * i) * CW + h * ON + j), v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) sum[i][h][j + k] = r ? sum[i][h][j + k] + v[k] : v[k];
              }
            }
          done_run();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (ok && grp + GR * i < NCH) do_item(grp + GR * i, 0, sum[i][0], sum[i][PAIR ? 1 : 0]);
      } else {
        if (!wait_run()) break;
        const uint32_t tacc = tbase + (run & 1u) * BN + lane_base;
#pragma unroll 1
        for (int c = grp; c < NCH && ok; c += GR) do_item(c, tacc, nullptr, nullptr);
        if (!ok) break;
        done_run();
      }
    }
    if (!ok && lane == 0) atomicExch(&bars->abort_, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == S::kEpiWarps + 1) {
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
  Mat A, B;
  int major;
  bool gated, f32;  // f32: fp32 operands (in terms) and outputs
  int epi, cfg;  // cfg: 0: CG 2, 1: CG 1 x BN 128, 2: CG 1 x BN 64
};

bool tensor_map_3d(CUtensorMap* m, const Mat& x, int esize, int box_cols, int box_rows);
bool run_fwd_product(const Product& p, cudaStream_t s);   // K-major, bf16 operands
bool run_e4m3_product(const Product& p, cudaStream_t s);  // K-major, e4m3 operands
bool run_dz_product(const Product& p, cudaStream_t s);
bool run_grad_product(const Product& p, cudaStream_t s);  // MN-major operands

template <int CG, int BN, int MAJOR, int KIND, bool GATED, int EPI, class TO, bool PROMOTE>
bool launch_tc(const Product& p, cudaStream_t s) {
  using S = Shape<CG, BN, GATED, EPI, TO>;
  auto* kernel = tc_kernel<CG, BN, MAJOR, KIND, GATED, EPI, TO, PROMOTE>;
  static int grid_max[64] = {};  // (host threads may race on it: each computes the same value)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
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
  TcArgs a = p.a;
  a.by_splits = make_div(uint32_t(a.splits));
  a.by_batch = make_div(uint32_t(a.mt) * uint32_t(a.nt));
  a.by_group = make_div(8u * uint32_t(a.nt));
  a.by_last = make_div(a.mt % 8 ? uint32_t(a.mt % 8) : 8u);
  const long long g = units * CG < grid_max[dev] ? units * CG : grid_max[dev];
  cfg.gridDim = dim3(unsigned(g));
  constexpr int es = KIND == kBf16 ? 2 : 1;
  CUtensorMap mA, mB;
  if (!tensor_map_3d(&mA, p.A, es, MAJOR == kNN ? 64 : 128 / es, MAJOR == kNN ? 64 : 128)) return false;
  if (!tensor_map_3d(&mB, p.B, es, MAJOR != kKK ? 64 : 128 / es,
                     MAJOR != kKK ? 64 : (GATED && CG == 1 ? BN / 2 : BN / CG)))
    return false;
  return cudaLaunchKernelEx(&cfg, kernel, a, mA, mB) == cudaSuccess;
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
