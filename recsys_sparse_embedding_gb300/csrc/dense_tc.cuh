// The matrix products of the dense operators on the tensor cores: D = A B^T
// with the operator's epilogue, sums in fp32.
//
// One persistent, warp-specialised kernel. A work unit is a tile of 128 CG x
// BN accumulators (CG CTAs of a cluster work on one tile together: CG = 2
// halves what each SM has to read of B), over all of K or one K-split.
//   the load warp  brings A and B by TMA: K-blocks of 128 bytes per row in the
//            128-byte swizzle, through a ring of stages;
//   the MMA warp  issues the MMAs (tcgen05.mma, in the cluster's first CTA)
//            into one of two accumulators in tensor memory;
//   16 (or 8) epilogue warps  turn the other accumulator into outputs, in
//            items of 32 rows (a warp's lane quarter, one row per lane) by 32
//            columns. Inputs (the residual, or the upstream gradient; loaded
//            an item ahead) and outputs change between a row per lane and 16
//            bytes of neighbouring lanes in a 2 or 4 KB buffer per warp, so
//            that global memory sees whole row segments. (Not by TMA: its
//            stores and loads queue behind the operands' loads, 2 us an item.)
// So a tile's loads, MMAs and epilogue overlap the next tile's. Operands come
// as three-dimensional tensors [plane][row][column]:
//   - K-major (columns are K) or MN-major (rows are K: W in dx = dz W, both
//     operands in dW = dz^T x, which needs no transposed copies);
//   - planes: the three bf16 terms of an fp32 operand, and the gate and up
//     halves of a gated layer (both in one tile of the forward; two segments
//     of K in dx; two batches in dW).
//
// fp32 operands (F32): x = x1 + x2 + x3 exactly, each term the leading 8
// significant bits of what is left. x y is the sum of the terms' products;
// those below 2^-21 of it (x2 y3, x3 y2, x3 y3) are dropped. A K-block's three
// terms of A and of B are loaded once and multiplied six ways: x1 y1 into one
// accumulator, the five smaller products into another. TWO: the same with two terms,
// each rounded to nearest (x to 2^-17), and the three products x1 y1, x1 y2, x2 y1 in
// one accumulator: half the work, for results that are not kept in fp32.
//
// Runs. The tensor cores truncate each addition to an accumulator towards zero.
// Measured, a sum of n additions (K / 16) is low by 0.5 n 2^-25 of itself where
// the terms' signs are random, by 0.9 (n = 64) to 3 n 2^-25 (n = 2^14 and more)
// where they are alike, and by less where terms are zero, so no factor gives it
// back. Where fp32 results depend on it, the accumulator takes a run of K-blocks
// at a time, and the epilogue warps add the runs up in registers, rounding to
// nearest: runs of 4 K-blocks in fp32, and of 8 in the z from which a bf16
// backward sums db (gated, 16384 x 1024 -> 4096: db is off by 5.2e-7 of its
// 2-norm, 1.1e-6 with all of K in one run, and no more at longer K: 2.4e-6 at
// 2048 in one run). Its tiles are then 256 x 128, so that a tile's sums fit the
// registers: the product and db's column sums take 229 us instead of 196.
// (256 x 256 with sums in registers spills: 310 us against 290 in a version
// whose MMA loop was slower.) Other products take all of
// a unit's K in one run: their outputs are rounded to bf16, and K is split before
// its runs grow long enough to be seen there.
//
// Measured in a graph over changing operands, bf16: gated forward of 16384 x
// 1024 -> 4096 142 us (1.93 PFLOP/s; the tensor pipe is busy 91% of the launch).
// 8192 x 4096 -> 1024 42.5 us, 45.5 with the residual (1.62 and 1.51 PFLOP/s:
// 128 tiles on 76 CTA pairs are two waves, 84% filled), in e4m3 25.3 and 27.9.
// fp32 8192 x 256 -> 512 18.3 us with its operands' laying out. 8192 x 512 ->
// 256 6.1 us: latency, one tile per CTA.
//
// Every wait is bounded; one that runs out sets DSF_FLAG_TIMEOUT.
#pragma once
#include <cuda.h>
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
namespace dense {

// What the epilogue does with an accumulator.
enum Epi {
  kEpiFwd = 0,   // out = act(z), or act(z) * z' for a gated layer
  kEpiRes = 4,   // out = in + act(z): the forward with a residual
  kEpiDz = 1,    // out = dz (planes dg, du for a gated layer; fp32: its three
                 // terms) from in = dy; column sums
  kEpiOut = 2,   // out = the accumulator
  kEpiPart = 3,  // fp32 partial sums of a K-split: plane split * planes + (half or batch); kDual: job 0 only
  kEpiAcc = 5,   // the same, added to what the planes hold
  // operands of the next product (TWO: in two terms, else in three):
  kEpiTerms = 8,  // out = the accumulator's terms; in fp32 too where f32 is given
  kEpiPoly = 9,   // out = the terms of c0 [row = column] + c1 in + c2 times the accumulator
  // softmax cross entropy over the columns (z in units of log 2 where it is an
  // exponent; the target's column per row):
  kEpiLse = 6,   // per row a reference and the sum of exp(z - it), over the tiles that a warp has of the row; z of the target
  kEpiXent = 7,  // out = g (exp(z - lse) - [column = target]) (fp32: its three terms); column sums
};
enum Kind { kBf16 = 0, kE4m3 = 1 };
// A and B K-major; B MN-major; both; two products in one launch, job 0 with
// both MN-major (dW), job 1 with B (dx)
enum Major { kKK = 0, kKN = 1, kNN = 2, kDual = 3 };

// Division of unsigned 32-bit numbers by a fixed divisor (Granlund and
// Montgomery, Division by invariant integers using multiplication): q = (mulhi(n, m) + n) >> l
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

// One product: its tiles, its operands' planes, its output.
struct Job {
  int M, N;          // rows; output columns (a gated layer's: F)
  int mt, nt, nb;    // tiles along M and N, batches (halves of dW)
  Div by_splits, by_batch, by_group, by_last;  // splits; mt nt; 8 nt; M tiles of the last group of 8
  int nkb, kbps;     // K-blocks per segment, per split
  int splits, nseg;  // K-splits; segments of K (the halves in dx)
  // planes: A: term * a_term + segment * a_seg + batch; B: term * b_term +
  // segment (a gated layer's: twice that, + half)
  int a_term, a_seg, b_term;
  void* out;
  long long ldo, out_plane;  // strides in elements
  int out_vec;               // rows at 16-byte boundaries
};

struct TcArgs {
  Job job[2];
  // kDual: the job with the longer units goes first, dealt round; `rest` of the
  // clusters have one unit of it more than the others (h0 and h0 - 1), and the
  // other job's units are dealt (l0 and l1 to each) so that the sums agree
  int first, rest, h0, l0, l1;
  int act;
  const float *bias, *xs, *ws;  // z = acc * xs[m] * ws[n] + bias[n] (each nullable; the up half at n + N)
  const void* in;               // kEpiRes, kEpiDz, kEpiAcc, kEpiPoly
  long long ldi;
  int in_vec;   // rows at 16-byte boundaries
  float* part;  // kEpiDz, kEpiXent: column sums of 32 rows each, [ceil(M / 32)][halves * N] (nullable)
  const long long* target;  // kEpiLse, kEpiXent: per row the target's column in all of W (outside: none)
  int v0;                   // the first column here, of them
  float2* stat;             // kEpiLse: [slot * warps per row + warp][M] (reference, sum); a lane's slot: its first N tile of the row
  // kEpiLse, kEpiXent: gm neighbouring M tiles are worked on together, each by
  // `lanes` clusters that share out its N tiles; so a cluster stays with its rows,
  // and a tile of B serves gm tiles of A from L2
  int gm, lanes, positions;  // positions: N tiles times groups of gm
  Div by_nt;
  float* zt;                // kEpiLse: [M]
  const float2* rows;       // kEpiXent: [M] (lse, g)
  float* f32;               // kEpiTerms: rows of ldo elements (nullable)
  float c0, c1, c2;         // kEpiPoly
  int tri;                  // kEpiPart: 0, or the tiles of a symmetric product that touch its lower triangle (tri_tiles)
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
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An arrival that orders nothing but itself: what it announces (accumulators
// and bias read) is complete in registers. A release would wait for the
// thread's global stores.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
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
template <int CG, int BN, int MAJOR, bool GATED, int EPI, bool F32>
struct Shape {
  using TO = typename std::conditional<F32 || EPI == kEpiPart || EPI == kEpiAcc || EPI == kEpiTerms || EPI == kEpiPoly, float,
                                       __nv_bfloat16>::type;  // input and output
  static constexpr int ON = GATED ? BN / 2 : BN;  // output columns per tile
  // Epilogue warps: four per lane quarter (scheduler). Two where the kernel
  // needs the registers (168 instead of 96 a thread: a gated dz, whose items
  // hold 64 sums or outputs each), which in fp32 is also all that 64 columns
  // have work for.
  static constexpr int kEpiWarps = GATED && ((F32 && EPI != kEpiPart) || EPI == kEpiDz) ? 8 : 16;
  static constexpr int kGroups = kEpiWarps / 4;
  static constexpr int kLoad = kEpiWarps, kMma = kEpiWarps + 1;
  static constexpr int kThreads = 32 * (kEpiWarps + 2);
  static constexpr int ITEM = 32 * 32 * int(sizeof(TO));
  static constexpr int BNC = BN / CG;  // B rows (or MN-major columns) in this CTA
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BNC * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int EBYTES = kEpiWarps * ITEM;
  static constexpr bool BIAS = EPI == kEpiFwd || EPI == kEpiRes || EPI == kEpiDz || EPI == kEpiLse || EPI == kEpiXent;
  // bias floats of an item that each epilogue warp keeps in shared memory (the
  // gated forward's six stages leave room for the gate's alone; the up half's
  // are handed round by shuffles)
  static constexpr int BIAS_N = !BIAS ? 0 : (GATED && kEpiWarps == 8 ? 64 : 32);
  static constexpr int BIAS_BYTES = kEpiWarps * BIAS_N * 4, BAR_BYTES = 256;
  static constexpr int kRoom = 227 * 1024 - EBYTES - BIAS_BYTES - BAR_BYTES;
  static constexpr int STAGES = kRoom / STAGE < 8 ? kRoom / STAGE : 8;
  static constexpr int SMEM = STAGES * STAGE + EBYTES + BIAS_BYTES + BAR_BYTES;
  static constexpr int ACC = F32 ? 2 * BN : BN;  // tensor-memory columns of an accumulator
  // K-blocks per accumulator run (0: all of a unit's), and accumulators
  static constexpr int RUN = F32 ? 4 : (EPI == kEpiDz && BN < 256 ? 8 : 0);
  static constexpr uint32_t NACC = !F32 && RUN ? 4 : 2;
  static constexpr uint32_t TCOLS = NACC * ACC;
  static_assert(TCOLS <= 512 && (TCOLS & (TCOLS - 1)) == 0, "tensor memory columns");
  static_assert(STAGES >= 4, "ring");
  // A successor that is started early, and waits for this kernel, must not hold
  // tensor memory that a block here has yet to allocate.
  static_assert(SMEM > 114 * 1024, "one block per SM");
  static_assert(B_BYTES % (GATED && CG == 1 ? 2048 : 1024) == 0, "swizzle atoms");
};

struct Bars {
  uint64_t full[8], empty[8], tfull[4], tempty[4];
  uint32_t tmem;
  int abort_;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

constexpr float kFar = 3e38f;  // (for infinity where differences have to stay defined: no reference; the lse of a row left out)
// References of sums of exponentials lie within this of zero, in units of log 2: z log2 e -
// reference is then off by at most 64 where the reference was rounded, which the exponentials'
// range bears and the reference takes back. A logit farther below adds nothing, as -inf
// (masks of -1e9 or of the type's lowest value); one farther above makes the sum infinite.
constexpr float kFarthest = 0x1p30f;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// The leading 8 significant bits of x, as bf16 bits in the upper half of the
// word; x becomes what is left (of a non-finite x, a NaN).
__device__ __forceinline__ uint32_t take_term(float& x) {
  const uint32_t h = __float_as_uint(x) & 0xffff0000u;
  x -= __uint_as_float(h);
  return h;
}

// sums of 32 columns over a warp's 32 rows (one row per lane): lane l returns
// column l's. Each step halves the columns a lane holds.
__device__ __forceinline__ float column_sum(const float* v, int lane) {
  float t[16];
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float lo = w == 16 ? v[i] : t[i], hi = w == 16 ? v[i + 16] : t[(i + w) & 15];
      t[i] = (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, w);
    }
  }
  return t[0];
}

__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  tmem_ld16(t, v);
  tmem_ld16(t + 16, v + 16);
}

// Byte `at` of row r of a 32-row buffer with ROWB bytes per row: 16-byte slots
// XOR-swizzled by the row, so that neither a slot of 8 rows nor whole rows
// meet in a bank.
template <int ROWB>
__device__ __forceinline__ int slot(int r, int at) {
  return r * ROWB + (((at >> 4) ^ (ROWB == 64 ? (r >> 1) & 3 : r & 7)) << 4) + (at & 15);
}


// ---------------------------------------------------------------- the kernel
template <int CG, int BN, int MAJOR, int KIND, bool GATED, int EPI, bool F32, bool TWO>
__global__ void __launch_bounds__(Shape<CG, BN, MAJOR, GATED, EPI, F32>::kThreads, 1)
    tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap mapA,
              const __grid_constant__ CUtensorMap mapB, const __grid_constant__ CUtensorMap mapA1,
              const __grid_constant__ CUtensorMap mapB1) {
  using S = Shape<CG, BN, MAJOR, GATED, EPI, F32>;
  using TO = typename S::TO;
  constexpr bool DUAL = MAJOR == kDual, BMN = MAJOR != kKK;
  constexpr int kBK = KIND == kBf16 ? 64 : 128;  // K elements per block (128 bytes)
  constexpr int ON = S::ON, CW = 32, STAGES = S::STAGES, TERMS = F32 ? 3 : (TWO ? 2 : 1), RUN = S::RUN;
  static_assert(!(GATED && BMN), "a gated layer's product is K-major");
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sE = sm + STAGES * S::STAGE;
  float* sBias = reinterpret_cast<float*>(sE + S::EBYTES);
  Bars* bars = reinterpret_cast<Bars*>(sE + S::EBYTES + S::BIAS_BYTES);
  if (smem_u32(sm) & 1023u) {  // (the swizzle atoms' alignment; every thread of the grid takes the same way)
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, DSF_FLAG_TIMEOUT);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int unit0 = blockIdx.x / CG, units_step = gridDim.x / CG;

  if (warp == S::kLoad && lane == 0) {
    prefetch_map(&mapA);
    prefetch_map(&mapB);
    if (DUAL) {
      prefetch_map(&mapA1);
      prefetch_map(&mapB1);
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < int(S::NACC); ++i) {
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
  if (warp != S::kLoad) {
    if (warp == S::kMma) {
      tmem_alloc_cg<CG>(&bars->tmem, S::TCOLS);
      tmem_relinquish_cg<CG>();
      tc_fence_before();
    }
    asm volatile("bar.sync 1, %0;" ::"n"(S::kThreads - 32) : "memory");
    tc_fence_after();
    tbase = bars->tmem;
  }
  volatile int* aborted = &bars->abort_;

  // The cluster's i-th unit; false after the last. In a product: split-minor,
  // then N tiles within groups of M tiles, so that the units in flight share
  // rows of A and of B in L2.
  struct Unit {
    int job, m0, n0, batch, split, kb0, kbn;
  };
  const int lane_of = EPI == kEpiLse || EPI == kEpiXent ? unit0 / a.gm : 0, mg = unit0 - lane_of * a.gm;
  const auto& job0 = a.job[0];
  const bool tri = EPI == kEpiPart && !DUAL && a.tri != 0;
  const int units = (tri ? a.tri : job0.mt * job0.nt * job0.nb) * job0.splits;
  auto unit_at = [&](int i, Unit& t) {
    int u = unit0 + i * units_step;
    t.job = 0;
    if (DUAL) {
      const bool more = unit0 < a.rest;
      const int h = a.h0 - (more ? 0 : 1), j = i - h;
      t.job = j < 0 ? a.first : 1 - a.first;
      if (j >= 0) {
        if (j >= (more ? a.l0 : a.l1)) return false;
        u = more ? j * a.rest + unit0 : a.rest * a.l0 + j * (units_step - a.rest) + unit0 - a.rest;
        const Job& o = a.job[t.job];
        if (u >= o.mt * o.nt * o.nb * o.splits) return false;
      }
    } else if (EPI == kEpiLse || EPI == kEpiXent) {
      const int at = lane_of + i * a.lanes;
      if (lane_of >= a.lanes || at >= a.positions) return false;
      const int group = int(div_by(at, a.by_nt)), m = group * a.gm + mg;
      if (m >= job0.mt) return false;
      t.split = t.batch = 0;
      t.m0 = m * 128 * CG + int(rank) * 128;
      t.n0 = (at - group * job0.nt) * ON;
      t.kb0 = 0;
      t.kbn = job0.nkb;
      return true;
    } else if (u >= units) {
      return false;
    }
    const Job& o = a.job[DUAL ? t.job : 0];
    uint32_t r = div_by(u, o.by_splits);
    t.split = u - int(r) * o.splits;
    if (tri) {  // M tile m has its first Q (m + 1) N tiles
      constexpr int Q = 128 * CG / ON;
      int m = int((sqrtf(8.f / Q * float(r) + 1.f) - 1.f) * 0.5f);
      if (Q * m * (m + 1) / 2 > int(r)) --m;
      if (Q * (m + 1) * (m + 2) / 2 <= int(r)) ++m;
      t.batch = 0;
      t.m0 = m * 128 * CG + int(rank) * 128;
      t.n0 = (int(r) - Q * m * (m + 1) / 2) * ON;
      t.kb0 = t.split * o.kbps;
      t.kbn = min(o.kbps, o.nkb - t.kb0);
      return true;
    }
    t.batch = int(div_by(r, o.by_batch));
    r -= uint32_t(t.batch) * o.by_batch.d;
    const uint32_t grp = div_by(r, o.by_group);
    r -= grp * o.by_group.d;
    const bool whole = int(grp * 8 + 8) <= o.mt;
    const uint32_t n = whole ? r >> 3 : div_by(r, o.by_last), gm = whole ? 8 : o.by_last.d;
    t.m0 = int(grp * 8 + r - n * gm) * 128 * CG + int(rank) * 128;
    t.n0 = int(n) * ON;
    t.kb0 = t.split * o.kbps;
    t.kbn = min(o.kbps, o.nkb - t.kb0);
    return true;
  };

  if (warp == S::kLoad) {
    // ------------------------------------------------ loads (one thread)
    if (lane == 0) {
      pdl_wait();
      uint32_t it = 0, st = 0, lap = 0;  // stages filled so far; the next stage, and the ring's laps before it
      bool ok = true;
      const uint32_t full0 = CG == 2 ? mapa(smem_u32(&bars->full[0]), 0) : smem_u32(&bars->full[0]);
      Unit t;
      for (int i = 0; ok && unit_at(i, t); ++i) {
        const Job& o = a.job[DUAL ? t.job : 0];
        const bool amn = MAJOR == kNN || (DUAL && t.job == 0);
        const void* ma = DUAL && t.job ? &mapA1 : &mapA;
        const void* mb = DUAL && t.job ? &mapB1 : &mapB;
        for (int sg = 0; sg < o.nseg && ok; ++sg)
          for (int k = 0; k < t.kbn && ok; ++k)
#pragma unroll 1
            for (int term = 0; term < TERMS; ++term) {
              if (lap && !(ok = mbar_wait(&bars->empty[st], (lap - 1) & 1u))) break;
              const int za = term * o.a_term + sg * o.a_seg + t.batch, zb = term * o.b_term + sg;
              const uint32_t bar = full0 + uint32_t(st) * 8u;
              if (rank == 0) mbar_arrive_expect_tx(&bars->full[st], uint32_t(CG * S::STAGE));
              const uint32_t sa = smem_u32(sm + st * S::STAGE), sb = sa + S::A_BYTES;
              const int kx = (t.kb0 + k) * kBK;
              if (amn) {
                tma_load_3d<CG>(sa, ma, t.m0, kx, za, bar);
                tma_load_3d<CG>(sa + 8192, ma, t.m0 + 64, kx, za, bar);
              } else {
                tma_load_3d<CG>(sa, ma, kx, t.m0, za, bar);
              }
              if (GATED) {
                if (CG == 2) {  // the gate half in one CTA, the up half in the other
                  tma_load_3d<CG>(sb, mb, kx, t.n0, 2 * zb + int(rank), bar);
                } else {
                  tma_load_3d<CG>(sb, mb, kx, t.n0, 2 * zb, bar);
                  tma_load_3d<CG>(sb + S::B_BYTES / 2, mb, kx, t.n0, 2 * zb + 1, bar);
                }
              } else if (BMN) {
#pragma unroll
                for (int j = 0; j < S::BNC / 64; ++j)
                  tma_load_3d<CG>(sb + j * 8192, mb, t.n0 + int(rank) * S::BNC + 64 * j, kx, zb, bar);
              } else {
                tma_load_3d<CG>(sb, mb, kx, t.n0 + int(rank) * S::BNC, zb, bar);
              }
              ++it;
              if (++st == uint32_t(STAGES)) st = 0, ++lap;
            }
      }
      // the last loads have landed before the CTA may end (bounded)
      if (!ok) atomicExch(&bars->abort_, 1);
      for (uint32_t j = it > uint32_t(STAGES) ? it - STAGES : 0; rank == 0 && j < it; ++j)
        if (!mbar_wait(&bars->full[j % STAGES], (j / STAGES) & 1u)) atomicExch(&bars->abort_, 1);
    }
    __syncwarp();
  } else if (warp == S::kMma) {
    // ------------------------------------------------ MMAs (one thread of the cluster)
    // (The warp runs the loop together and one elected lane issues: descriptors
    // then stay in uniform registers. A K-block of 256 x 128 takes 0.22 us, by a
    // loop of one lane 0.29.)
    if (rank == 0) {
      pdl_wait();  // (its waits are bounded, what the stream does before is not)
      const bool lead = elect_one();
      constexpr uint32_t ID = (1u << 4) | (KIND == kBf16 ? (1u << 7) | (1u << 10) : 0u) | (BMN ? 1u << 16 : 0u) |
                              (uint32_t(BN >> 3) << 17) | (uint32_t((128 * CG) >> 4) << 24);
      uint32_t run = 0, st = 0, phase = 0;  // the next stage, and its barrier's phase
      bool ok = true;
      const uint32_t s0 = smem_u32(sm);
      bool amn = MAJOR == kNN;
      const uint64_t db0 = BMN ? mn_desc(s0 + S::A_BYTES) : sw128_kmajor_desc(s0 + S::A_BYTES);
      // a K-block of A in stage sa times one of B in stage sb (addresses in the
      // descriptors count 16 bytes)
      auto block = [&](uint32_t d, uint32_t sa, uint32_t sb, bool accumulate) {
        const uint64_t da = (amn ? mn_desc(s0) : sw128_kmajor_desc(s0)) + sa * uint32_t(S::STAGE >> 4),
                       db = db0 + sb * uint32_t(S::STAGE >> 4);
        const uint32_t id = ID | (amn ? 1u << 15 : 0u), step = amn ? 128 : 2;
        if (!lead) return;
#pragma unroll
        for (uint32_t kk = 0; kk < 4; ++kk)
          mma<CG, KIND>(d, da + kk * step, db + kk * (BMN ? 128 : 2), id, (accumulate || kk > 0) ? 1u : 0u);
      };
      auto take = [&](uint32_t& stage) {  // the next stage, once it is filled
        stage = st;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[st], phase));
        if (++st == uint32_t(STAGES)) st = 0, phase ^= 1u;
        tc_fence_after();
        return ok;
      };
      Unit t;
      for (int i = 0; ok && unit_at(i, t); ++i) {
        if (DUAL) amn = t.job == 0;
        for (int left = a.job[DUAL ? t.job : 0].nseg * t.kbn; left > 0 && ok; ++run) {
          const int len = RUN ? min(left, RUN) : left;
          const uint32_t acc = run % S::NACC, d = tbase + acc * S::ACC;
          if (run >= S::NACC &&
              !(ok = __all_sync(0xffffffffu, mbar_wait(&bars->tempty[acc], (run / S::NACC - 1) & 1u))))
            break;
          tc_fence_after();
          for (int k = 0; k < len; ++k) {
            uint32_t x, y, z;
            if (!take(x)) break;
            block(d, x, x, k > 0);
            if (TWO) {
              if (!take(y)) break;
              block(d, x, y, true);
              block(d, y, x, true);
            }
            if (F32) {
              if (!take(y)) break;
              block(d + BN, x, y, k > 0);
              block(d + BN, y, x, true);
              block(d + BN, y, y, true);
              if (!take(z)) break;
              block(d + BN, x, z, true);
              block(d + BN, z, x, true);
            }
            if (!lead) continue;
            mma_commit<CG>(&bars->empty[x]);
            if (F32 || TWO) mma_commit<CG>(&bars->empty[y]);
            if (F32) mma_commit<CG>(&bars->empty[z]);
          }
          if (ok && lead) mma_commit<CG>(&bars->tfull[acc]);
          left -= len;
        }
      }
      if (!ok && lead) atomicExch(&bars->abort_, 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue
    pdl_wait();
    const int q = warp & 3, grp = warp >> 2;
    uint8_t* buf = sE + warp * S::ITEM;
    float* wbias = sBias + warp * S::BIAS_N;
    const uint32_t lane_base = uint32_t(q * 32) << 16;
    constexpr bool FWD = EPI == kEpiFwd || EPI == kEpiRes, IN = EPI == kEpiRes || EPI == kEpiDz || EPI == kEpiAcc || EPI == kEpiPoly;
    constexpr bool XENT = EPI == kEpiLse || EPI == kEpiXent;
    constexpr bool SCALED = KIND == kE4m3 && FWD;
    // the item leaves as three (TWO: two) bf16 terms
    constexpr bool TERMS_OUT = (F32 && (EPI == kEpiDz || EPI == kEpiXent)) || EPI == kEpiTerms || EPI == kEpiPoly;
    constexpr bool PAIR = GATED && EPI != kEpiPart;   // an item takes gate and up accumulators
    constexpr int GR = S::kGroups, ROWB = CW * int(sizeof(TO));
    constexpr int halves = GATED ? 2 : 1;
    // items of a tile side by side: over its accumulators for a gated layer's partial sums, else over its outputs
    constexpr int NCH = (GATED && EPI == kEpiPart ? BN : ON) / CW;
    constexpr int NI = (NCH + GR - 1) / GR;  // items per warp and tile
    const bool has_bias = S::BIAS && a.bias;
    const TO* in0 = static_cast<const TO*>(a.in);
    auto in_of = [&](const Unit& t) {  // (kEpiAcc: the unit's plane)
      return EPI == kEpiAcc ? in0 + (t.split * job0.nb + t.batch) * job0.out_plane : in0;
    };
    const uint32_t tempty0 = CG == 2 ? mapa(smem_u32(&bars->tempty[0]), 0) : smem_u32(&bars->tempty[0]);

    // columns j .. j + 7 of this lane's row, from and to the buffer
    auto get8 = [&](int j, float* v) {
#pragma unroll
      for (int k = 0; k < int(sizeof(TO)) / 2; ++k) {
        const uint4 u = *reinterpret_cast<const uint4*>(buf + slot<ROWB>(lane, j * int(sizeof(TO)) + 16 * k));
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
    auto put8 = [&](int j, const float* v) {
#pragma unroll
      for (int k = 0; k < int(sizeof(TO)) / 2; ++k) {
        uint4 w;
        if (sizeof(TO) == 4)
          w = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                         __float_as_uint(v[4 * k + 3]));
        else
          w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        *reinterpret_cast<uint4*>(buf + slot<ROWB>(lane, j * int(sizeof(TO)) + 16 * k)) = w;
      }
    };
    auto put8_bf16 = [&](int j, const float* v) {  // (where TO is float)
      *reinterpret_cast<uint4*>(buf + slot<64>(lane, 2 * j)) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    };
    // A 16-byte piece of an item for each lane: 4 (bf16) or 8 (fp32) lanes side
    // by side on a row. Pieces past the matrix's edge element by element.
    constexpr int EL = 16 / int(sizeof(TO)), LPR = CW / EL, RPI = 32 / LPR, NV = 32 / RPI;
    const int piece_row = lane / LPR, piece_col = lane % LPR * EL;
    auto load_item = [&](const TO* in, uint4* v, int r0, int c0) {
      const int cc = c0 + piece_col;
      const TO* p0 = in + (long long)(r0 + piece_row) * a.ldi + cc;
      const long long step = RPI * a.ldi;
      if (r0 + 32 <= job0.M && c0 + CW <= job0.N) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p0 + i * step));
        return;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = r0 + i * RPI + piece_row;
        const TO* p = p0 + i * step;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r >= job0.M || cc >= job0.N) continue;
        if (cc + EL <= job0.N) {
          v[i] = __ldg(reinterpret_cast<const uint4*>(p));
        } else {
          uint32_t w[4] = {};
#pragma unroll
          for (int e = 0; e < EL - 1; ++e)
            if (cc + e < job0.N) {
              if (sizeof(TO) == 4) w[e] = __float_as_uint(to_float(p[e]));
              else w[e / 2] |= (__float_as_uint(to_float(p[e])) >> 16) << (16 * (e & 1));
            }
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    // the buffer's item (of element type T) to rows r0 .., columns c0 .. of base
    auto store_item = [&](const Job& o, auto* base, int r0, int c0) {
      using T = typename std::remove_pointer<decltype(base)>::type;
      constexpr int ES = int(sizeof(T)), RB = CW * ES, E = 16 / ES, L = CW / E, RP = 32 / L;
      __syncwarp();
      if (o.out_vec) {
        const int pr = lane / L, pc = lane % L * E, cc = c0 + pc;
        if (r0 + 32 <= o.M && c0 + CW <= o.N) {
          T* p = base + (long long)(r0 + pr) * o.ldo + cc;
          const long long step = RP * o.ldo;
#pragma unroll
          for (int i = 0; i < 32 / RP; ++i)
            *reinterpret_cast<uint4*>(p + i * step) = *reinterpret_cast<const uint4*>(buf + slot<RB>(i * RP + pr, pc * ES));
          __syncwarp();
          return;
        }
#pragma unroll
        for (int i = 0; i < 32 / RP; ++i) {
          const int rr = i * RP + pr, r = r0 + rr;
          const uint8_t* b = buf + slot<RB>(rr, pc * ES);
          T* p = base + (long long)r * o.ldo + cc;
          if (r >= o.M || cc >= o.N) continue;
          if (cc + E <= o.N) {
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(b);
          } else {
            for (int e = 0; cc + e < o.N; ++e) p[e] = reinterpret_cast<const T*>(b)[e];
          }
        }
      } else {
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
          if (r0 + r < o.M && c0 + lane < o.N)
            base[(long long)(r0 + r) * o.ldo + c0 + lane] = *reinterpret_cast<const T*>(buf + slot<RB>(r, lane * ES));
      }
      __syncwarp();
    };
    // What the warp's next item ((unit, item) pairs in order) takes from memory:
    // its columns' bias, one column per lane; its input, where it can be loaded
    // in pieces: bf16 into registers; fp32, whose sums take the registers, as
    // far as L2.
    constexpr bool PRE = IN && sizeof(TO) == 2;
    uint4 pin[PRE ? NV : 1];
    float bias_g = 0.f, bias_u = 0.f;
    const bool ahead = IN || (XENT ? has_bias : S::BIAS);  // whether items take anything from memory
    auto prefetch = [&](bool any, const Unit& t, int c) {
      if (!ahead) return;
      const int r = any ? t.m0 + 32 * q : job0.M, cc = t.n0 + c * CW;
      const TO* in = in_of(t);
      if (PRE) load_item(in, pin, a.in_vec ? r : job0.M, cc);
      if (IN && !(PRE && a.in_vec) && r + lane < job0.M && cc < job0.N) {
        const TO* p = in + (long long)(r + lane) * a.ldi + cc;
        prefetch_l2(p);
        prefetch_l2(p + min(CW, job0.N - cc) - 1);  // (unaligned rows: perhaps another line)
      }
      if (S::BIAS) {
        const bool there = any && has_bias && cc + lane < job0.N;
        bias_g = there ? __ldg(a.bias + cc + lane) : 0.f;
        if (GATED) bias_u = there ? __ldg(a.bias + job0.N + cc + lane) : 0.f;
      }
    };
    auto prefetch_after = [&](int i, const Unit& t, int c) {  // the item after item c of unit i
      if (!ahead) return;
      if (c + GR < NCH) {
        prefetch(true, t, c + GR);
      } else {
        Unit n;
        n.m0 = n.n0 = n.split = n.batch = 0;
        prefetch(unit_at(i + 1, n) && grp < NCH, n, grp);
      }
    };
    Unit t;
    t.m0 = t.n0 = t.split = t.batch = 0;
    prefetch(unit_at(0, t) && grp < NCH, t, grp);
    uint32_t run = 0;
    bool ok = true;
    auto wait_run = [&]() {  // the run's accumulator is complete
      if (*aborted) ok = false;
      if (ok && lane == 0) ok = mbar_wait(&bars->tfull[run % S::NACC], (run / S::NACC) & 1u);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after();
      return ok;
    };
    auto done_run = [&]() {  // and may be overwritten
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(tempty0 + (run % S::NACC) * 8u);
      ++run;
    };
    // a cross entropy's rows: the target's column (or one that no item has), lse and
    // g; kEpiLse: the reference (in units of log 2) and sum over the warp's items so
    // far, written when the warp goes on to other rows
    int stat_m0 = -1, stat_slot = 0, tgt = -1;
    float2 of_row = make_float2(0.f, 0.f);
    bool fresh = true;
    float top = -kFarthest, total = 0.f;
    auto put_stat = [&]() {
      const int r = stat_m0 + 32 * q + lane;
      if (stat_m0 >= 0 && r < job0.M) a.stat[((long long)stat_slot * GR + grp) * job0.M + r] = make_float2(top, total);
    };
    for (int i = 0; ok && unit_at(i, t); ++i) {
      const Job& jb = a.job[DUAL ? t.job : 0];
      const int row0 = t.m0 + 32 * q, row = row0 + lane;
      const TO* in = in_of(t);
      if (XENT && t.m0 != stat_m0) {  // other rows: their targets, lse and g
        if (EPI == kEpiLse) put_stat();
        stat_m0 = t.m0;
        stat_slot = t.n0 / ON;
        fresh = true;
        top = -kFarthest, total = 0.f;
        const long long id = row < jb.M ? __ldg(a.target + row) : -1, d = id - a.v0;
        tgt = id >= 0 && d >= 0 && d < jb.N ? int(d) : -1;
        if (EPI == kEpiXent) of_row = row < jb.M ? __ldg(a.rows + row) : make_float2(0.f, 0.f);
      }
      // one item: 32 rows by CW columns. In runs: pg, pu hold its sums
      auto do_item = [&](int c, uint32_t tacc, float* pg, float* pu) {
        const int cc = GATED && EPI == kEpiPart ? (c * CW) % ON : c * CW, col0 = t.n0 + cc;
        if (row0 >= jb.M || col0 >= jb.N) {
          prefetch_after(i, t, c);
          return;
        }
        // g (and up): the accumulators of this lane's row, then the outputs. (Their
        // loads run while the item's other inputs are laid out.)
        float g_[32], up_[PAIR ? 32 : 1];
        float* g = g_;
        float* up = up_;
        if (RUN) {
          g = pg;
          up = pu;
        } else {
          tmem_ld32(tacc + uint32_t(c * CW), g);
          if (PAIR) tmem_ld32(tacc + uint32_t(c * CW) + ON, up);
        }
        if (S::BIAS) {
          wbias[lane] = bias_g;
          if (S::BIAS_N == 64) wbias[32 + lane] = bias_u;
          if (!IN) __syncwarp();
        }
        if (IN) {
          if (a.in_vec) {
            if (!PRE) {
              uint4 v[NV];
              load_item(in, v, row0, col0);
#pragma unroll
              for (int i = 0; i < NV; ++i)
                *reinterpret_cast<uint4*>(buf + slot<ROWB>(i * RPI + piece_row, piece_col * int(sizeof(TO)))) = v[i];
            } else {
#pragma unroll
              for (int i = 0; i < NV; ++i)
                *reinterpret_cast<uint4*>(buf + slot<ROWB>(i * RPI + piece_row, piece_col * int(sizeof(TO)))) =
                    pin[PRE ? i : 0];
            }
          } else {  // one column per lane, RB rows in flight
            constexpr int RB = S::kEpiWarps == 8 ? 32 : 16;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += RB) {
              TO v[RB];
#pragma unroll
              for (int r = 0; r < RB; ++r) {
                v[r] = TO(0.f);
                if (row0 + r0 + r < jb.M && col0 + lane < jb.N) v[r] = in[(long long)(row0 + r0 + r) * a.ldi + col0 + lane];
              }
#pragma unroll
              for (int r = 0; r < RB; ++r)
                *reinterpret_cast<TO*>(buf + slot<ROWB>(r0 + r, lane * int(sizeof(TO)))) = v[r];
            }
          }
          __syncwarp();
        }
        const float bu = bias_u;
        prefetch_after(i, t, c);  // (a whole item's time ahead)
        // e4m3: the row's scale, and the columns' (one per lane, handed round by shuffles)
        float xs = 0.f, ws = 0.f, wsu = 0.f;
        if (SCALED) {
          if (row < jb.M) xs = __ldg(a.xs + row);
          if (col0 + lane < jb.N) {
            ws = __ldg(a.ws + col0 + lane);
            if (PAIR) wsu = __ldg(a.ws + jb.N + col0 + lane);
          }
        }
        if (!RUN) tmem_ld_wait();
        if (XENT) {
          const float* b = wbias;
          if (has_bias)
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(b + j);
            float2 lo = make_float2(g[j], g[j + 1]), hi = make_float2(g[j + 2], g[j + 3]);
            lo = lo + make_float2(f.x, f.y);
            hi = hi + make_float2(f.z, f.w);
            g[j] = lo.x, g[j + 1] = lo.y, g[j + 2] = hi.x, g[j + 3] = hi.y;
          }
          const bool target_here = __any_sync(0xffffffffu, unsigned(tgt - col0) < 32u);
          if constexpr (EPI == kEpiLse) {
            if (col0 + CW > jb.N) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (col0 + k >= jb.N) g[k] = -INFINITY;
            }
            if (target_here) {
              float z = 0.f;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (tgt - col0 == k) z = g[k];
              if (unsigned(tgt - col0) < 32u && row < jb.M) a.zt[row] = z;
            }
            // Any reference serves that keeps the sum in range: the first item's
            // maximum, until a sum grows past 2^80 (or is none)
            auto add = [&](float ref) {
              float2 s[2] = {pair(0.f), pair(0.f)};
#pragma unroll
              for (int k = 0; k < 32; k += 4)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float2 e = __ffma2_rn(make_float2(g[k + 2 * h], g[k + 2 * h + 1]), pair(kLog2e), pair(-ref));
                  s[h] = s[h] + make_float2(exp2_fast(e.x), exp2_fast(e.y));
                }
              return (s[0].x + s[0].y) + (s[1].x + s[1].y);
            };
            float more = 0.f;
            if (!fresh) more = total + add(top);
            const bool anew = fresh || !(more < 0x1p80f);  // (row by row: a row's bits depend on no other's)
            if (__any_sync(0xffffffffu, anew)) {
              float m[4];  // (fmaxf leaves a NaN to the sum)
#pragma unroll
              for (int k = 0; k < 4; ++k) m[k] = fmaxf(fmaxf(g[k], g[k + 4]), g[k + 8]);
#pragma unroll
              for (int k = 12; k < 32; k += 4)
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], g[k + e]);
              const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
              const float now = fmaxf(top, fminf(most * kLog2e, kFarthest));
              const float again = total * exp2_fast(top - now) + add(now);
              if (anew) more = again, top = now;
              fresh = false;
            }
            total = more;
            __syncwarp();  // (the bias is read)
            return;
          } else {
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 e = __ffma2_rn(make_float2(g[k], g[k + 1]), pair(kLog2e), pair(-of_row.x));
            const float2 p = make_float2(exp2_fast(e.x), exp2_fast(e.y)) * pair(of_row.y);
            g[k] = p.x, g[k + 1] = p.y;
          }
          if (of_row.y == 0.f) {  // (a row left out, whatever it holds)
#pragma unroll
            for (int k = 0; k < 32; ++k) g[k] = 0.f;
          }
          if (target_here) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (tgt - col0 == k) g[k] -= of_row.y;
          }
          if (col0 + CW > jb.N) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (col0 + k >= jb.N) g[k] = 0.f;
          }
          }
        }
        // eight columns at a time, from the accumulators to the buffer
        auto math = [&](auto act_tag) {
          constexpr int ACT = decltype(act_tag)::value;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float* v = g + j;
            float* w = up + (PAIR ? j : 0);
            if (SCALED) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[k] *= xs * __shfl_sync(0xffffffffu, ws, j + k);
                if (PAIR) w[PAIR ? k : 0] *= xs * __shfl_sync(0xffffffffu, wsu, j + k);
              }
            }
            float x[8];
            if (IN) get8(j, x);
            float b[8], d[8];  // (16 bytes a time: shared memory is what the MMAs run on)
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
              if (S::BIAS && !XENT) *reinterpret_cast<float4*>(b + k) = *reinterpret_cast<const float4*>(wbias + j + k);
              if (PAIR && S::BIAS_N == 64)
                *reinterpret_cast<float4*>(d + k) = *reinterpret_cast<const float4*>(wbias + 32 + j + k);
            }
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              if (EPI == kEpiAcc) v[k] += x[k], v[k + 1] += x[k + 1];
              if (EPI == kEpiPoly)
#pragma unroll
                for (int e = k; e < k + 2; ++e) v[e] = fmaf(a.c2, v[e], a.c1 * x[e]) + (row == col0 + j + e ? a.c0 : 0.f);
              if (!S::BIAS || XENT) continue;
              const float2 b2 = make_float2(b[k], b[k + 1]);
              float2 z = make_float2(v[k], v[k + 1]);
              z = z + b2;
              float2 y = pair(0.f);
              if (PAIR) {
                y = make_float2(w[PAIR ? k : 0], w[PAIR ? k + 1 : 0]);
                if (S::BIAS_N == 64)
                  y = y + make_float2(d[k], d[k + 1]);
                else
                  y = y + make_float2(__shfl_sync(0xffffffffu, bu, j + k), __shfl_sync(0xffffffffu, bu, j + k + 1));
              }
              const float2 in2 = make_float2(x[k], x[k + 1]);
              if (FWD) {
                z = act_value<ACT>(z);
                if (PAIR) z = z * y;
                if (EPI == kEpiRes) z = z + in2;
              } else {
                float2 value, slope;
                act_both<ACT>(z, value, slope);
                z = (PAIR ? in2 * y : in2) * slope;
                if (PAIR) y = in2 * value;
              }
              v[k] = z.x, v[k + 1] = z.y;
              if (PAIR) w[PAIR ? k : 0] = y.x, w[PAIR ? k + 1 : 0] = y.y;
            }
            if (DUAL && EPI == kEpiPart && !F32 && t.job) put8_bf16(j, v);
            else if (!TERMS_OUT) put8(j, v);
          }
        };
        if (FWD || EPI == kEpiDz) {
          switch (a.act) {
            case DSF_ACT_RELU: math(std::integral_constant<int, DSF_ACT_RELU>{}); break;
            case DSF_ACT_SILU: math(std::integral_constant<int, DSF_ACT_SILU>{}); break;
            case DSF_ACT_GELU: math(std::integral_constant<int, DSF_ACT_GELU>{}); break;
            default: math(std::integral_constant<int, DSF_ACT_NONE>{});
          }
        } else {
          math(std::integral_constant<int, DSF_ACT_NONE>{});
        }
        auto sums = [&](const float* v, int half) {
          const float s = column_sum(v, lane);
          if (col0 + lane < jb.N) a.part[((long long)(row0 >> 5) * halves + half) * jb.N + col0 + lane] = s;
        };
        if (TERMS_OUT) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(jb.out);
#pragma unroll
          for (int h = 0; h < halves; ++h) {
            float* v = h ? up : g;
            if (a.part) sums(v, h);
            __syncwarp();  // (the input is read, or the last term gone, before the buffer is written)
            if (EPI == kEpiTerms && a.f32) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) put8(j, v + j);
              store_item(jb, a.f32, row0, col0);
            }
#pragma unroll
            for (int term = 0; term < (TWO ? 2 : 3); ++term) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (TWO) {
                    float* e = v + j + 2 * k;
                    w[k] = pack_bf16x2(e[0], e[1]);
                    e[0] -= __uint_as_float(w[k] << 16), e[1] -= __uint_as_float(w[k] & 0xffff0000u);
                    continue;
                  }
                  const uint32_t lo = take_term(v[j + 2 * k]), hi = take_term(v[j + 2 * k + 1]);
                  w[k] = __byte_perm(lo, hi, 0x7632);
                }
                *reinterpret_cast<uint4*>(buf + slot<64>(lane, 2 * j)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
              store_item(jb, o + (term * halves + h) * jb.out_plane, row0, col0);
            }
          }
        } else {
          // (two products: only job 0 has partial sums)
          const bool part = EPI == kEpiAcc || (EPI == kEpiPart && (!DUAL || t.job == 0));
          int plane = t.batch;
          if (part) plane = GATED ? t.split * 2 + (c * CW) / ON : t.split * jb.nb + t.batch;
          TO* o = static_cast<TO*>(jb.out) + plane * jb.out_plane;
          if (DUAL && EPI == kEpiPart && !F32 && !part)
            store_item(jb, static_cast<__nv_bfloat16*>(jb.out) + plane * jb.out_plane, row0, col0);
          else
            store_item(jb, o, row0, col0);
          if (EPI == kEpiDz && PAIR) {  // du takes the buffer after dg has left it
#pragma unroll
            for (int j = 0; j < 32; j += 8) put8(j, up + (PAIR ? j : 0));
            store_item(jb, o + jb.out_plane, row0, col0);
          }
          if ((EPI == kEpiDz || EPI == kEpiXent) && a.part) {
            sums(g, 0);
            if (PAIR) sums(up, 1);
          }
        }
      };
      if constexpr (RUN > 0) {
        float sum[NI][PAIR ? 2 : 1][32];
        const int runs = (jb.nseg * t.kbn + RUN - 1) / RUN;
        for (int r = 0; r < runs; ++r) {
          if (!wait_run()) break;
          const uint32_t tacc = tbase + (run % S::NACC) * S::ACC + lane_base;
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
              if (grp + GR * i >= NCH) continue;
              const uint32_t col = tacc + uint32_t((grp + GR * i) * CW + h * ON);
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                float v[16], w[16];
                tmem_ld16(col + j, v);
                if (F32) tmem_ld16(col + BN + j, w);  // the smaller products
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) sum[i][h][j + k] = (r ? sum[i][h][j + k] : 0.f) + (F32 ? v[k] + w[k] : v[k]);
              }
            }
          done_run();
        }
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < NI; ++k)
          if (grp + GR * k < NCH) do_item(grp + GR * k, 0, sum[k][0], sum[k][PAIR ? 1 : 0]);
      } else {
        if (!wait_run()) break;
        const uint32_t tacc = tbase + (run % S::NACC) * S::ACC + lane_base;
#pragma unroll 1
        for (int c = grp; c < NCH; c += GR) do_item(c, tacc, nullptr, nullptr);
        done_run();
      }
    }
    if constexpr (EPI == kEpiLse) put_stat();
    if (!ok && lane == 0) atomicExch(&bars->abort_, 1);
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == S::kMma) {
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

// One product.
struct Product {
  TcArgs a;
  Mat A, B, A1, B1;  // kDual: job 1's
  int major;
  bool gated, f32, two;  // f32: fp32 operands (in three terms); two: in two terms
  int epi, cfg;     // cfg: 0: CG 2, 1: CG 1 x BN 128, 2: CG 1 x BN 64, 3 (bf16 dz in runs): CG 2 x BN 128
  long long weight[2];  // kDual: a unit's time, by job
  int* lse_slots;       // kEpiLse: where the launch writes how many slots a row has
};

bool tensor_map_3d(CUtensorMap* m, const Mat& x, int esize, int box_cols, int box_rows);
// Launches; false: a launch or a tensor map failed.
bool run_fwd_product(const Product& p, cudaStream_t s);   // K-major, bf16 operands
bool run_e4m3_product(const Product& p, cudaStream_t s);  // K-major, e4m3 operands
bool run_dz_product(const Product& p, cudaStream_t s);
bool run_grad_product(const Product& p, cudaStream_t s);  // MN-major operands
bool run_dual_product(const Product& p, cudaStream_t s);
bool run_xent_product(const Product& p, cudaStream_t s);  // kEpiLse, kEpiXent: configurations 0 and 1
bool run_acc_product(const Product& p, cudaStream_t s);   // kEpiAcc, B MN-major
bool run_two_product(const Product& p, cudaStream_t s);   // operands in two terms: kEpiPart, any one Major
bool run_terms_product(const Product& p, cudaStream_t s);  // kEpiTerms, kEpiPoly (K-major): operands in two or three terms

// How two products' units go to C clusters: the longer units dealt round (to
// the first `rest` clusters h0, to the others h0 - 1), the others so that
// every cluster's time comes near the mean. w: a unit's time, by job; load:
// the most of any.
struct Deal {
  int first, rest, h0, l0, l1;
  long long load;
};
inline Deal deal(const TcArgs& a, const long long (&w)[2], long long C) {
  long long n[2];
  for (int j = 0; j < 2; ++j) n[j] = (long long)a.job[j].mt * a.job[j].nt * a.job[j].nb * a.job[j].splits;
  const int f = w[0] >= w[1] ? 0 : 1;
  const long long N = n[f], L = n[1 - f], W = w[f], V = w[1 - f];
  const long long h0 = (N + C - 1) / C, rest = N - (h0 - 1) * C, others = C - rest;
  const long long mean = (N * W + L * V + C - 1) / C, near = mean > h0 * W ? (mean - h0 * W) / V : 0;
  Deal best{f, int(rest), int(h0), 0, 0, INT64_MAX};
  for (long long t = near; t <= near + 1; ++t) {  // the mean from below, or from above
    long long l0 = others > 0 ? t : (L + rest - 1) / rest;
    if (l0 * rest > L) l0 = (L + rest - 1) / rest;
    const long long left = L > rest * l0 ? L - rest * l0 : 0, l1 = others > 0 ? (left + others - 1) / others : 0;
    const long long x = h0 * W + l0 * V, y = others > 0 ? (h0 - 1) * W + l1 * V : 0;
    if ((x > y ? x : y) < best.load) {
      best.l0 = int(l0);
      best.l1 = int(l1);
      best.load = x > y ? x : y;
    }
  }
  return best;
}

// A cross entropy's groups: of 4 M tiles, or fewer where those would leave more clusters
// without work, by 3 of 100 at least per choice (a tile of B is read from memory once per
// group: more than 2 are enough). So single tiles may be taken up to 93 (of 96 in groups of
// 4, 3 of 100 are none), groups of 4 are from there on.
inline int lse_group(long long mt, long long clusters) {
  int best = 1;
  double most = 0;
  for (int gm = 4; gm >= 1; gm /= 2) {
    if (gm > clusters) continue;
    const double e = double(mt) / double((mt + gm - 1) / gm * gm) * double(clusters / gm * gm) / double(clusters);
    if (e > most + 0.03) best = gm, most = e;
  }
  return best;
}

// Slots times rows that M rows' pairs have room for (growing with M): a slot for every
// cluster up to those 93 tiles, for a quarter of them beyond. A launch has no more lanes
// than slots (or than N tiles: a lane without one has no pair).
constexpr long long kLseClusters = 152, kLseSingle = 93 * 128;
inline long long lse_room(long long M) {
  const long long m = M < kLseSingle ? M : kLseSingle;
  return m * kLseClusters + (M - m) * (kLseClusters / 4);
}

template <int CG, int BN, int MAJOR, int KIND, bool GATED, int EPI, bool F32, bool TWO = false>
bool launch_tc(const Product& p, cudaStream_t s) {
  using S = Shape<CG, BN, MAJOR, GATED, EPI, F32>;
  auto* kernel = tc_kernel<CG, BN, MAJOR, KIND, GATED, EPI, F32, TWO>;
  static std::atomic<int> grid_max[64];  // (host threads may race on it: each computes the same value)
  int dev = 0;
  if (!succeeded(cudaGetDevice(&dev)) || dev < 0 || dev >= 64) return false;
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
  int most = grid_max[dev].load(std::memory_order_acquire);
  if (most == 0) {
    int sms = 0, n = 0;
    if (!succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM)) ||
        !succeeded(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
      return false;
    if (CG == 2) {
      cfg.gridDim = dim3(unsigned(sms / 2 * 2));
      if (!succeeded(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) || n < 1) return false;
      most = 2 * n;
    } else {
      most = sms;
    }
    grid_max[dev].store(most, std::memory_order_release);
  }
  TcArgs a = p.a;
  long long n[2] = {0, 0};  // units
  for (int j = 0; j < (MAJOR == kDual ? 2 : 1); ++j) {
    Job& o = a.job[j];
    n[j] = (long long)(EPI == kEpiPart && MAJOR != kDual && a.tri ? a.tri : (long long)o.mt * o.nt * o.nb) * o.splits;
    if (n[j] <= 0 || n[j] * CG > INT32_MAX) return false;
    o.by_splits = make_div(uint32_t(o.splits));
    o.by_batch = make_div(uint32_t(o.mt) * uint32_t(o.nt));
    o.by_group = make_div(8u * uint32_t(o.nt));
    o.by_last = make_div(o.mt % 8 ? uint32_t(o.mt % 8) : 8u);
  }
  const long long want = (n[0] + n[1]) * CG, g = want < most ? want : most;
  if (MAJOR == kDual) {
    const Deal d = deal(a, p.weight, g / CG);
    a.first = d.first;
    a.rest = d.rest;
    a.h0 = d.h0;
    a.l0 = d.l0;
    a.l1 = d.l1;
  }
  if (EPI == kEpiLse || EPI == kEpiXent) {
    const Job& o = a.job[0];
    a.gm = lse_group(o.mt, g / CG);
    a.lanes = int(g / CG / a.gm);
    const long long room = lse_room(o.M) / o.M;  // (what binds only where the device has more clusters)
    if (EPI == kEpiLse && o.nt > room && a.lanes > room) a.lanes = int(room);
    a.by_nt = make_div(uint32_t(o.nt));
    const long long positions = (long long)((o.mt + a.gm - 1) / a.gm) * o.nt;
    if (positions + a.lanes > INT32_MAX) return false;
    a.positions = int(positions);
    if (EPI == kEpiLse) *p.lse_slots = o.nt < a.lanes ? o.nt : a.lanes;
  }
  cfg.gridDim = dim3(unsigned(g));
  constexpr int es = KIND == kBf16 ? 2 : 1;
  constexpr bool amn = MAJOR == kNN || MAJOR == kDual;
  CUtensorMap mA, mB, mA1, mB1;
  if (!tensor_map_3d(&mA, p.A, es, amn ? 64 : 128 / es, amn ? 64 : 128)) return false;
  if (!tensor_map_3d(&mB, p.B, es, MAJOR != kKK ? 64 : 128 / es,
                     MAJOR != kKK ? 64 : (GATED && CG == 1 ? BN / 2 : BN / CG)))
    return false;
  mA1 = mA;
  mB1 = mB;
  if (MAJOR == kDual && (!tensor_map_3d(&mA1, p.A1, es, 64, 128) || !tensor_map_3d(&mB1, p.B1, es, 64, 64))) return false;
  return succeeded(cudaLaunchKernelEx(&cfg, kernel, a, mA, mB, mA1, mB1));
}

// Tile configurations: accumulator columns (an fp32 product's wide tiles are
// half as wide: it holds two sets) and rows.
constexpr int cfg_bn(int cfg, bool f32) { return cfg == 0 ? (f32 ? 128 : 256) : (cfg == 2 ? 64 : 128); }
constexpr int cfg_rows(int cfg) { return cfg % 3 == 0 ? 256 : 128; }

template <int MAJOR, int KIND, bool GATED, int EPI, bool F32>
bool launch_cfg(const Product& p, cudaStream_t s) {
  if (p.cfg == 0) return launch_tc<2, cfg_bn(0, F32), MAJOR, KIND, GATED, EPI, F32>(p, s);
  if (p.cfg == 1) return launch_tc<1, 128, MAJOR, KIND, GATED, EPI, F32>(p, s);
  if constexpr (EPI == kEpiDz && !F32)
    if (p.cfg == 3) return launch_tc<2, 128, MAJOR, KIND, GATED, EPI, F32>(p, s);
  if constexpr (!GATED) return launch_tc<1, 64, MAJOR, KIND, GATED, EPI, F32>(p, s);
  return false;
}

}  // namespace dense
}  // namespace dsf
