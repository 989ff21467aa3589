// The cross entropy where x and W are narrow (bf16, K <= 128): the rows' sums, dx and
// dW in one pass each that computes the logits and keeps nothing of them.
//
// A block has 128 rows of one matrix (x for the sums and dx, W for dW) in shared
// memory and streams the other's by 128: S = rows times streamed rows on the tensor
// cores. 16 warps add up exp(S - reference) per row (the sums); or they turn S into
// dz = g (exp(z - lse) - [target]), rounded to bf16, in tensor memory in S's own
// place, and dz times the streamed rows (the same shared memory, now MN-major) is
// added to the block's output in tensor memory. dz in memory instead costs 6 bytes
// a logit (written, read twice): at K = 64 that took 7.9 of a training step's 10.1
// ms (8192 rows, 846,812 columns).
//
//   load warp   TMA: the block's rows once per unit, then the streamed tiles, with
//               what the epilogue takes per column (bias, or lse, g and target)
//   MMA warps   one for S, one for dz times its rows: each waits for its own operands
//               only (one warp for both, in turn, took 1290 cycles a tile of waiting)
//   16 epilogue warps in two sets: even tiles and odd ones. A warp has 32 rows (a
//               tensor-memory quarter) by 64 columns of its tiles.
//
// Tensor memory: three S buffers of 128 columns, so that a set finds its next tile's
// S there when it has done one; then the output's columns. No unit is full (8192 rows and
// 131,072 columns of 64, under ncu 273 us for the sums, 263 for dx, 336 for dW): the
// exponentials take 512 cycles a tile (32 ex2 a clock and SM, measured on their own), 44,
// 47 and 39% of the time; the tensor pipe is busy 22, 47 and 38%, the issue slots 55 to
// 61%, and in dW's pass shared memory's read path 70% (lse, g and target per column). An
// SM's 19 warps wait on what they issued themselves: results, tensor memory, branches.
// (Registers are all taken, 96 a thread; ptxas reports 116 to 120 bytes of spill stores for
// dW's pass, 20 for dx's.) Slower or no faster:
// dz in buffers of its own in tensor memory or in shared memory, S given back as soon
// as it is in registers (they spill more), 24 epilogue warps, four S buffers for the sums.
// At K = 256 dz in memory was faster (both gradients 1.6 ms against 1.9).
// Sums of a unit are at most 512 tiles (65536 terms) long; dx is split over the
// columns anyway (planes, added in order by finish_kernel). Every wait is bounded.
#pragma once
#include "dense_tc.cuh"

namespace dsf {
namespace dense {

enum XentMode { kSums = 0, kDx = 1, kDw = 2 };

struct PassArgs {
  int R, C;             // the blocks' rows, the streamed rows
  int rt, ct;           // tiles of 128 of them
  int chunks, per;      // chunks of the streamed tiles, tiles in one
  int K;
  // per streamed row, in whole tiles of 128: kSums, kDx: bias (nullable); kDw: lse in
  // units of log 2 (kFar where a row is left out or past the end), g, target
  const float *col0, *col1;
  const int* col_id;
  // per row of the block: kDx: lse, g; kDw: bias (nullable)
  const float *row0, *row1;
  const long long* target;  // kSums, kDx
  void* out;            // dW bf16 [R][K] (nullable); dx fp32 [chunks][R][ldo]
  long long ldo, plane;
  float* db;            // kDw: [4][R] sums of dz (nullable)
  float2* stat;         // kSums: [4 chunks][R] (reference, sum)
  float* zt;            // kSums: [R] the target's logit
  int* status;
};

template <int NK>
struct PassShape {
  static constexpr int kWarps = 16, kLoad = 16, kMma = 17, kMma2 = 18;
  static constexpr int threads(int mode) { return mode == kSums ? 32 * 18 : 32 * 19; }  // (the sums have one product)
  static constexpr int TILE = NK * 16384;
  static constexpr int COLS = 3 * 512;  // a stage's values per column
  // Buffers of the block's rows: with two, a unit's are there before the one before it
  // ends, and its streamed tiles are not held up (K > 64: the room is better spent on
  // those).
  static constexpr int RB = NK == 1 ? 2 : 1;
  static constexpr int kRoom = 227 * 1024 - RB * TILE - 512;
  static constexpr int STAGES = kRoom / (TILE + COLS) < 8 ? kRoom / (TILE + COLS) : 8;
  static constexpr int SMEM = (STAGES + RB) * TILE + STAGES * COLS + 512;
  static constexpr int NB = 3;  // S buffers
  static_assert(STAGES >= NB && NB * 128 + NK * 64 <= 512, "tiles under way; tensor memory");
  static_assert(STAGES >= 2 && SMEM > 114 * 1024, "ring; one block per SM");
};

struct PassBars {
  uint64_t full[8], empty[8], rows_full[2], rows_empty[2], s_full[3], p_full[3], acc_full, acc_empty;
  uint32_t tmem;
  int abort_;
};
static_assert(sizeof(PassBars) <= 512, "barrier block");

// MN-major operand of 128 K indices per 64 columns (mn_desc's has 64)
__device__ __forceinline__ uint64_t mn_desc_128(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFFu) | uint64_t(16384u >> 4) << 16 | uint64_t(1024u >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}

template <int MODE, int NK>
__global__ void __launch_bounds__(PassShape<NK>::threads(MODE), 1)
    xent_pass_kernel(const __grid_constant__ PassArgs a, const __grid_constant__ CUtensorMap map_rows,
                     const __grid_constant__ CUtensorMap map_stream) {
  using S = PassShape<NK>;
  constexpr int STAGES = S::STAGES, NB = S::NB, COLS = S::COLS, RB = S::RB;
  constexpr bool DW = MODE == kDw;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* s_rows = sm + STAGES * S::TILE;
  uint8_t* s_cols = s_rows + RB * S::TILE;
  PassBars* bars = reinterpret_cast<PassBars*>(s_cols + STAGES * COLS);
  if (smem_u32(sm) & 1023u) {  // (the swizzle atoms' alignment; every thread of the grid takes the same way)
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, DSF_FLAG_TIMEOUT);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == S::kLoad && lane == 0) {
    prefetch_map(&map_rows);
    prefetch_map(&map_stream);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < RB; ++i) {
      mbar_init(&bars->rows_full[i], 1);
      mbar_init(&bars->rows_empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 8);
    }
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->acc_empty, S::kWarps);
    bars->abort_ = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  pdl_go();
  uint32_t tbase = 0;
  if (warp == S::kMma) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  tbase = bars->tmem;
  volatile int* aborted = &bars->abort_;
  pdl_wait();

  // the block's i-th unit: rows [128 r, ...) over the chunk's tiles. Neighbouring
  // blocks have neighbouring rows of one chunk, so that its tiles come from L2.
  const int units = a.rt * a.chunks;
  struct Unit {
    int r0, c0, n, chunk;  // first row, first streamed tile, tiles
  };
  auto unit_at = [&](int i, Unit& t) {
    const int u = int(blockIdx.x) + i * int(gridDim.x);
    if (u >= units) return false;
    t.chunk = u / a.rt;
    t.r0 = (u - t.chunk * a.rt) * 128;
    t.c0 = t.chunk * a.per;
    t.n = min(a.per, a.ct - t.c0);
    return true;
  };

  if (warp == S::kLoad) {
    // ------------------------------------------------ loads (one thread)
    if (lane == 0) {
      bool ok = true;
      uint32_t it = 0;
      int i = 0;  // (units whose rows are asked for)
      Unit t;
      while (ok && unit_at(i, t)) {
        uint64_t* rows_full = &bars->rows_full[i % RB];
        uint8_t* rows = s_rows + i % RB * S::TILE;
        if (i >= RB && !(ok = mbar_wait(&bars->rows_empty[i % RB], (i / RB - 1) & 1))) break;
        ++i;
        mbar_arrive_expect_tx(rows_full, S::TILE);
#pragma unroll
        for (int k = 0; k < NK; ++k)
          tma_load_3d<1>(smem_u32(rows + k * 16384), &map_rows, k * 64, t.r0, 0, smem_u32(rows_full));
        for (int j = 0; j < t.n; ++j, ++it) {
          const uint32_t st = it % STAGES, lap = it / STAGES;
          if (lap && !(ok = mbar_wait(&bars->empty[st], (lap - 1) & 1u))) break;
          mbar_arrive_expect_tx(&bars->full[st], S::TILE + (DW ? 3 * 512 : (a.col0 ? 512 : 0)));
          const long long at = (long long)(t.c0 + j) * 128;
          if (DW || a.col0) bulk_g2s(s_cols + st * COLS, a.col0 + at, 512, &bars->full[st]);
          if (DW) {
            bulk_g2s(s_cols + st * COLS + 512, a.col1 + at, 512, &bars->full[st]);
            bulk_g2s(s_cols + st * COLS + 1024, a.col_id + at, 512, &bars->full[st]);
          }
#pragma unroll
          for (int k = 0; k < NK; ++k)
            tma_load_3d<1>(smem_u32(sm + st * S::TILE + k * 16384), &map_stream, k * 64, (t.c0 + j) * 128, 0,
                           smem_u32(&bars->full[st]));
        }
      }
      if (!ok) atomicExch(&bars->abort_, 1);
      // the last loads have landed before the block may end (bounded)
      for (int k = max(i - RB, 0); k < i; ++k)
        if (!mbar_wait(&bars->rows_full[k % RB], (k / RB) & 1)) atomicExch(&bars->abort_, 1);
      for (uint32_t j = it > uint32_t(STAGES) ? it - STAGES : 0; j < it; ++j)
        if (!mbar_wait(&bars->full[j % STAGES], (j / STAGES) & 1u)) atomicExch(&bars->abort_, 1);
    }
    __syncwarp();
  } else if (warp == S::kMma || warp == S::kMma2) {
    // ------------------------------------------------ MMAs (a warp together, one lane issues)
    const bool lead = elect_one();
    constexpr uint32_t ID1 = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(128 >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    constexpr uint32_t ID2 = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(NK * 64 >> 3) << 17) |
                             (uint32_t(128 >> 4) << 24);
    const uint32_t s0 = smem_u32(sm), acc = tbase + NB * 128;
    bool ok = true;
    uint32_t it = 0;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, phase & 1u));
      tc_fence_after();
      return ok;
    };
    auto done = [&](uint32_t t) {  // (the sums) tile t has been read
      if (wait(&bars->p_full[t % NB], t / NB) && lead) tc_commit(&bars->empty[t % STAGES]);
    };
    Unit t;
    for (int i = 0; ok && unit_at(i, t); ++i) {
      if (MODE == kSums || warp == S::kMma) {
        if (!wait(&bars->rows_full[i % RB], uint32_t(i / RB))) break;
        const uint64_t da = sw128_kmajor_desc(smem_u32(s_rows) + i % RB * S::TILE);
        for (int j = 0; j < t.n; ++j, ++it) {
          const uint32_t st = it % STAGES;
          if (!wait(&bars->full[st], it / STAGES)) break;
          // (S's buffer holds dz of tile it - NB until that has been multiplied)
          if (it >= NB && !wait(&bars->empty[(it - NB) % STAGES], (it - NB) / STAGES)) break;
          if (lead) {
            const uint64_t db = sw128_kmajor_desc(s0 + st * S::TILE);
#pragma unroll
            for (uint32_t k = 0; k < 4 * NK; ++k)
              mma<1, kBf16>(tbase + (it % NB) * 128, da + (k >> 2) * 1024 + (k & 3) * 2,
                            db + (k >> 2) * 1024 + (k & 3) * 2, ID1, k > 0);
            tc_commit(&bars->s_full[it % NB]);
          }
          if (MODE == kSums && j >= NB - 1) done(it - (NB - 1));
        }
        if (MODE == kSums)
          for (int j = max(t.n - (NB - 1), 0); ok && j < t.n; ++j) done(it - (t.n - j));
        if (ok && lead) tc_commit(&bars->rows_empty[i % RB]);
      } else {
        // dz of the tile times its rows
        for (int j = 0; j < t.n; ++j, ++it) {
          const uint32_t st = it % STAGES;
          if (!wait(&bars->full[st], it / STAGES) || !wait(&bars->p_full[it % NB], it / NB)) break;
          if (j == 0 && i > 0 && !wait(&bars->acc_empty, uint32_t(i - 1))) break;
          if (!lead) continue;
          const uint64_t db = mn_desc_128(s0 + st * S::TILE);
#pragma unroll
          for (uint32_t k = 0; k < 8; ++k)
            tc_mma_f16_ts(acc, tbase + (it % NB) * 128 + (k >> 2) * 64 + (k & 3) * 8, db + k * 128, ID2, j > 0 || k > 0);
          tc_commit(&bars->empty[st]);
        }
        if (ok && lead) tc_commit(&bars->acc_full);
      }
    }
    if (!ok && lead) atomicExch(&bars->abort_, 1);
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp >> 2) & 1, set = warp >> 3;
    const uint32_t lane_base = uint32_t(q * 32) << 16, s_col = tbase + half * 64 + lane_base;
    bool ok = true;
    uint32_t it = 0;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (ok && !__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1u)))
        ok = __all_sync(0xffffffffu, !*aborted && mbar_wait(bar, phase & 1u));
      tc_fence_after();
      return ok;
    };
    Unit t;
    for (int i = 0; ok && unit_at(i, t); ++i) {
      const int row0 = t.r0 + 32 * q, row = row0 + lane;
      const bool some = row0 < a.R;  // whether the warp's rows are there
      float bias = 0.f, sum = 0.f, lse = 0.f, g = 0.f, top = -kFarthest;
      bool fresh = true;
      int tgt = -1;
      if (row < a.R) {
        if (DW) {
          if (a.row0) bias = __ldg(a.row0 + row);
        } else {
          const long long id = __ldg(a.target + row);
          tgt = id >= 0 && id < a.C ? int(id) : -1;
          if (MODE == kDx) lse = __ldg(a.row0 + row), g = __ldg(a.row1 + row);
        }
      }
      for (int j = 0; j < t.n; ++j, ++it) {
        if (int(it & 1) != set) continue;
        const uint32_t st = it % STAGES, b = it % NB;
        if (!wait(&bars->full[st], it / STAGES) || !wait(&bars->s_full[b], it / NB)) break;
        const uint32_t s_at = s_col + b * 128;
        const int c0 = (t.c0 + j) * 128 + half * 64;
        if (some) {
          float zz[2][32];
          tmem_ld32(s_at, zz[0]);
          tmem_ld_wait();
          tmem_ld32(s_at + 32, zz[1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* z = zz[h];
            if (h) tmem_ld_wait();
            const float* cl = reinterpret_cast<const float*>(s_cols + st * COLS) + half * 64 + 32 * h;
            const int c = c0 + 32 * h;
            if (DW) {
              const float2 b2 = pair(bias);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 l = *reinterpret_cast<const float4*>(cl + k), gg = *reinterpret_cast<const float4*>(cl + 128 + k);
                const float2 e0 = __ffma2_rn(make_float2(z[k], z[k + 1]) + b2, pair(kLog2e), make_float2(-l.x, -l.y));
                const float2 e1 = __ffma2_rn(make_float2(z[k + 2], z[k + 3]) + b2, pair(kLog2e), make_float2(-l.z, -l.w));
                const float2 p0 = make_float2(exp2_fast(e0.x), exp2_fast(e0.y)) * make_float2(gg.x, gg.y);
                const float2 p1 = make_float2(exp2_fast(e1.x), exp2_fast(e1.y)) * make_float2(gg.z, gg.w);
                z[k] = p0.x, z[k + 1] = p0.y, z[k + 2] = p1.x, z[k + 3] = p1.y;
              }
              // the columns whose target is one of the warp's rows
              const int id = reinterpret_cast<const int*>(cl)[256 + lane];
              // (few but in the tiles of popular rows of W)
              if (__any_sync(0xffffffffu, unsigned(id - row0) < 32u)) {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                  const volatile int* d = reinterpret_cast<const int*>(cl) + 256 + k;  // (one at a time: registers)
                  if (*d == row) z[k] -= cl[128 + k];
                }
              }
              if (a.db) {
                float2 s2 = pair(0.f);
#pragma unroll
                for (int k = 0; k < 32; k += 2) s2 = s2 + make_float2(z[k], z[k + 1]);
                sum += s2.x + s2.y;
              }
            } else {
              if (a.col0)
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 f = *reinterpret_cast<const float4*>(cl + k);
                const float2 z0 = make_float2(z[k], z[k + 1]) + make_float2(f.x, f.y),
                             z1 = make_float2(z[k + 2], z[k + 3]) + make_float2(f.z, f.w);
                z[k] = z0.x, z[k + 1] = z0.y, z[k + 2] = z1.x, z[k + 3] = z1.y;
              }
              if (c + 32 > a.C) {  // the end of the columns
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (c + k >= a.C) z[k] = -INFINITY;
              }
              const bool target_here = __any_sync(0xffffffffu, unsigned(tgt - c) < 32u);
              if (MODE == kSums) {
                if (target_here) {
                  float zt = 0.f;
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (tgt - c == k) zt = z[k];
                  if (unsigned(tgt - c) < 32u) a.zt[row] = zt;
                }
                // (as in dense_tc.cuh: any reference that keeps the sum in range)
                auto add = [&](float ref) {
                  float2 s2[2] = {pair(0.f), pair(0.f)};
#pragma unroll
                  for (int k = 0; k < 32; k += 4)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      const float2 x =
                          __ffma2_rn(make_float2(z[k + 2 * e], z[k + 2 * e + 1]), pair(kLog2e), pair(-ref));
                      s2[e] = s2[e] + make_float2(exp2_fast(x.x), exp2_fast(x.y));
                    }
                  return (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
                };
                float more = 0.f;
                if (!fresh) more = sum + add(top);
                const bool anew = fresh || !(more < 0x1p80f);
                if (__any_sync(0xffffffffu, anew)) {
                  float most = z[0];  // (fmaxf leaves a NaN to the sum)
#pragma unroll
                  for (int k = 1; k < 32; ++k) most = fmaxf(most, z[k]);
                  const float now = fmaxf(top, fminf(most * kLog2e, kFarthest)), again = sum * exp2_fast(top - now) + add(now);
                  if (anew) more = again, top = now;
                  fresh = false;
                }
                sum = more;
              } else {
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                  const float2 e = __ffma2_rn(make_float2(z[k], z[k + 1]), pair(kLog2e), pair(-lse));
                  const float2 p = make_float2(exp2_fast(e.x), exp2_fast(e.y)) * pair(g);
                  z[k] = p.x, z[k + 1] = p.y;
                }
                if (target_here) {
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (tgt - c == k) z[k] -= g;
                }
              }
            }
            if (MODE != kSums) {
              uint32_t p[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) p[k] = pack_bf16x2(z[2 * k], z[2 * k + 1]);
              tmem_st16(s_at + 16 * h, p);
            }
          }
          if (MODE != kSums) tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[b]);
      }
      if (MODE == kSums) {
        if (ok && row < a.R) a.stat[((long long)t.chunk * 4 + set * 2 + half) * a.R + row] = make_float2(top, sum);
        continue;
      }
      if (!ok || !wait(&bars->acc_full, uint32_t(i))) break;
      if (DW && a.db && row < a.R) a.db[(long long)(set * 2 + half) * a.R + row] = sum;
      // the output's columns, a quarter of them per warp of the rows
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int c = ((set * 2 + half) * NK + k) * 16;
        float v[16];
        tmem_ld16(tbase + NB * 128 + c + lane_base, v);
        tmem_ld_wait();
        if (row >= a.R || c >= a.K || !a.out) continue;
        if (DW) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (long long)row * a.ldo + c;
          if (c + 16 <= a.K && a.ldo % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(o + e) =
                  make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]),
                             pack_bf16x2(v[e + 6], v[e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c + e < a.K) o[e] = __float2bfloat16(v[e]);
          }
        } else {  // (rows of whole vectors)
          float* o = static_cast<float*>(a.out) + t.chunk * a.plane + (long long)row * a.ldo + c;
          if (g == 0.f) {  // (a row left out, whatever W holds)
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            if (c + e < a.K) *reinterpret_cast<float4*>(o + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->acc_empty);
    }
    if (!ok && lane == 0) atomicExch(&bars->abort_, 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kMma) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0 && bars->abort_ && a.status) atomicOr(a.status, DSF_FLAG_TIMEOUT);
}

// One of XentMode's passes over `chunks` chunks of the streamed tiles.
bool run_xent_pass(int mode, const PassArgs& a, const Mat& rows, const Mat& stream, cudaStream_t s);

}  // namespace dense
}  // namespace dsf
