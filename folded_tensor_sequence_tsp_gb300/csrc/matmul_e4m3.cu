// matmul_e4m3.cu - the product of two e4m3 matrices with fp32 scales for blocks of 128:
//     C[m][n] = sum over blocks kb of K  sa[m][kb] sb[n][kb]  sum over k in kb  a[m][k] b[n][k]
// both operands K-major, the inner sum on the tensor cores (tcgen05, kind::f8f6f4), the outer one in
// fp32 registers: the scales are arbitrary fp32 numbers, so a block's product has to leave tensor
// memory before it can be scaled and added.
//
// A CTA has 128 rows of one operand (P, the lanes of tensor memory) beside BN rows of the other (Q, its
// columns), 384 threads:
//   warp 0      TMA producer: 128-byte K blocks of P and Q into a ring of 128B-swizzled buffers
//   warp 1      issues a block's four MMAs (N = BN, K = 32) into one of two accumulators in tensor
//               memory, each block from zero
//   warps 2, 3  fetch the scales of P's and Q's rows for KS blocks at a time into shared memory
//   warps 4..11 take a finished accumulator, scale it and add it to the tile's sum in registers (BN / 2
//               values per thread), while the next block's MMAs run
//
// Large products: pairs of CTAs on tiles of 256 x 256 (cta_group::2, P = A, Q = B), persistent. Each CTA of a
// pair loads half of Q, so a block brings 32 KB to an SM instead of 48; at 64 bytes per cycle into an SM, and
// at the rate of its shared memory, the 48 would take half as long again as the 512 cycles of the MMAs. The
// sums leave through shared memory by TMA under the next tile.
//   8192 x 8192 x 4096, scales for tiles, bf16 out: 205 to 215 us from box to box, 2560 to 2680 TFLOP/s (tensor
//   pipe 55 % active). Bound by the warps that add: a block takes them 860 cycles (tensor memory loads, barriers
//   and scales among busy shared memory, 256 cycles of fp32 FMAs). The same loads and MMAs without the sums: 167 us.
//   The same with a scale per row of both and fp32 out: 305 us; 512 cycles of FMA, and 268 MB to write.
//   Added to what C holds, the sums are written by the warps, in the open: 11008 x 4096 x 8192 (dw) 725 us, and 400
//   without the addition, whose sums leave by TMA; 2816 x 1024 x 1000 47 and 15 us.
// Few rows or few tiles: P = B, Q = A, so that 16 to 128 rows of A fill a tile; a tile per CTA or, with the
// blocks of K split, per cluster of CTAs, which join their sums through distributed shared memory in a
// fixed order.
//   4 x 11008 x 4096: 11.8 us (3.8 TB/s of weights; 1 MMA in 50 slots); 5 us of it are launch, first
//   loads and the cluster's join. 48 x 4096 x 11008: 14.6 us.
#include <cooperative_groups.h>

#include <algorithm>

#include "extent.h"
#include "tile_walk.h"
#include "tsp_device.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr uint32_t P_BYTES = BM * BK;
// Row stride of the sums in shared memory: a quarter warp's accesses to two columns' rows hit all banks
constexpr int PART = BM + 4;

// PAIR: two CTAs on a tile of 256 x BN, each with 128 rows of P, half of Q's in its shared memory, and
// BN columns of sums.
template <int BN, bool COLS, bool PAIR>
struct Config {
  static constexpr uint32_t Q_BYTES = (PAIR ? BN / 2 : BN) * BK;
  static constexpr uint32_t STAGE_BYTES = P_BYTES + Q_BYTES;
  // small tiles leave room for two CTAs on an SM
  static constexpr int CTAS = BN <= 32 ? 2 : 1;
  static constexpr int STAGES = PAIR ? 4 : BN == 128 ? 5 : BN == 64 ? 8 : 5;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  // Scales of KS blocks of K are fetched together, BM + QS for each: of P's rows, and of Q's rows or of its one or
  // two blocks of 128. (Tile scales, 8192 x 8192 x 4096: 4 blocks 230 us, 8 206 us, 16 205 us, 32 225 us.)
  static constexpr int KS = COLS ? 8 : 16;
  static constexpr int QS = COLS ? BN : 4;
  static constexpr int SCALES = KS * (BM + QS);
  static constexpr size_t SCALE_BYTES = 2 * SCALES * 4;
  static constexpr size_t OUT_BYTES = PAIR ? 65536 : 0;  // a pair's sums on their way out: 32 KB for each warpgroup
  static constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * STAGE_BYTES + OUT_BYTES + SCALE_BYTES + 256;
};

struct Params {
  int rows_p, rows_q, nkb;
  const float* sp;  // scale of row r: sp[(r >> p_shift) * ld_sp + kb]
  long long ld_sp;
  int p_shift;
  const float* sq;
  long long ld_sq;
  void* c;
  long long ldc;
  int c_f32, accumulate;
  int tma_out;  // pairs: C is written by TMA (rows start and end on 16 bytes, nothing is added)
  int group_p;  // tile order of the persistent walk
  DevStatus* status;
  unsigned long long limit_ns;
};

template <int CH>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[CH]) {
  if constexpr (CH == 16) tmem_ld16(addr, r);
  else tmem_ld8(addr, r);
}
template <int CH>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[CH]) {
  if constexpr (CH == 16) tmem_ld_wait16(r);
  else tmem_ld_wait8(r);
}

__device__ __forceinline__ void put(const Params& p, long long at, float v) {
  if (p.c_f32) {
    float* c = static_cast<float*>(p.c) + at;
    *c = p.accumulate ? *c + v : v;
  } else {
    static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
  }
}

// COLS: Q has a scale for every row (a column of the tile), else one for 128 rows.
// TURNED: P = B and Q = A, C[q][p]; else C[p][q].
template <int BN, bool COLS, bool TURNED, bool PAIR>
__global__ void __launch_bounds__(THREADS, Config<BN, COLS, PAIR>::CTAS)
    matmul_e4m3_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_c, const Params p) {
  using cfg = Config<BN, COLS, PAIR>;
  constexpr int STAGES = cfg::STAGES, HALF = BN / 2, KS = cfg::KS, QS = cfg::QS;
  constexpr int CH = BN == 16 ? 8 : 16;  // columns per tensor memory load (32: 243 us instead of 208)
  // Where columns have a scale each, and there are enough: a thread holds four rows of every fourth pair of
  // columns, so that it needs a fourth of them from shared memory (8192 x 8192 x 4096: 505 -> 385 us).
  constexpr bool QUAD = COLS && BN >= 64;
  extern __shared__ uint8_t smem_raw[];
  // an offset, not a pointer made from a number: the compiler goes on knowing that this is shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_p = smem;
  uint8_t* s_q = smem + STAGES * P_BYTES;
  uint8_t* s_out = smem + STAGES * cfg::STAGE_BYTES;
  float* s_scale = reinterpret_cast<float*>(s_out + cfg::OUT_BYTES);  // [2][KS][BM + QS]
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_scale) + cfg::SCALE_BYTES);
  uint64_t* full = bars;                   // [STAGES] TMA landed
  uint64_t* empty = bars + STAGES;         // [STAGES] MMAs reading the stage are done
  uint64_t* acc_full = bars + 2 * STAGES;  // [2] a block's product is complete
  uint64_t* acc_empty = acc_full + 2;      // [2] it has been taken
  uint64_t* scale_full = acc_empty + 2;    // [2] the scales of KS blocks are there
  uint64_t* scale_empty = scale_full + 2;  // [2] they have been read
  uint64_t* drain = scale_empty + 2;       // [1] every MMA issued has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();  // of the CTAs on one tile
  const int ranks = (int)cluster.num_blocks();
  const int split = PAIR ? 1 : ranks;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int TILE_P = PAIR ? 2 * BM : BM;
  const int num_p = (p.rows_p + TILE_P - 1) / TILE_P;
  const int num_q = (p.rows_q + BN - 1) / BN;
  const int num_tiles = num_p * num_q;
  const int first_tile = blockIdx.x / ranks, tile_step = gridDim.x / ranks;
  const int kb0 = PAIR ? 0 : (int)((long long)p.nkb * rank / split);
  const int kb1 = PAIR ? p.nkb : (int)((long long)p.nkb * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], PAIR ? 2 * EPI_WARPS : EPI_WARPS);
      mbar_init(&scale_full[a], 2);
      mbar_init(&scale_empty[a], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_p);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, cfg::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, cfg::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster.sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  dependents_may_start();
  prior_kernel_done();

  WaitBound wb{p.status, p.limit_ns, abort_flag};

  // Registers: 384 threads start with 168 each, the most that three warps per scheduler leave; the
  // sums of a wide tile (128 of them per thread) need more. 4 x 56 + 8 x 224 = 12 x 168.
  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ producer
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) last_parity[s] = -1;
      bool ok = true;
      for (int tile = first_tile; ok && tile < num_tiles; tile += tile_step) {
        int tp, tq;
        tile_coords(tile, num_p, num_q, p.group_p, tp, tq);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_short(&empty[stage], phase ^ 1u, wb, SITE_E4M3_PRODUCER)) {
            ok = false;
            break;
          }
          if constexpr (PAIR) {
            // both CTAs' bytes count on the first one's barrier, whose MMA warp reads them
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * cfg::STAGE_BYTES);
            const uint32_t bar = cluster_addr(&full[stage], 0);
            tma_load_2d_pair(s_p + stage * P_BYTES, &tm_p, bar, kb * BK, tp * TILE_P + rank * BM);
            tma_load_2d_pair(s_q + stage * cfg::Q_BYTES, &tm_q, bar, kb * BK, tq * BN + rank * (BN / 2));
          } else {
            mbar_arrive_expect_tx(&full[stage], cfg::STAGE_BYTES);
            tma_load_2d(s_p + stage * P_BYTES, &tm_p, &full[stage], kb * BK, tp * BM);
            tma_load_2d(s_q + stage * cfg::Q_BYTES, &tm_q, &full[stage], kb * BK, tq * BN);
          }
#pragma unroll
          for (int s = 0; s < STAGES; ++s)
            if (s == stage) last_parity[s] = (int)phase;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Do not leave while something is on its way to this CTA's shared memory: a TMA copy or, from the MMA warp of a
      // pair's first CTA, an arrival of a commit. A stage whose empty barrier is through the phase of its last copy has
      // neither (its MMAs have read the copy), the sums have seen every product, and the drain is the last
      // commit. Where a wait gave up, copies of the first CTA are waited for at their own barriers, and the
      // second one gives its copies, which count there, a millisecond.
      WaitBound wd{p.status, p.limit_ns, nullptr};
      if constexpr (PAIR) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
          if (ok && last_parity[s] >= 0) ok = mbar_wait(&empty[s], (uint32_t)last_parity[s], wb, SITE_DRAIN);
        if (rank != 0) mbar_wait(drain, 0, wd, SITE_DRAIN);
      }
      if (PAIR && rank != 0) {
        if (!ok) {
          const unsigned long long t0 = global_ns();
          while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
        }
      } else if (!PAIR || !ok) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
          if (last_parity[s] >= 0) mbar_wait(&full[s], (uint32_t)last_parity[s], wd, SITE_DRAIN);
      }
    }
    if (warp == 1 && (!PAIR || rank == 0)) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = make_idesc_e4m3(TILE_P, BN);
      const uint64_t dp0 = make_sdesc_sw128(smem_addr(s_p), 16, 1024);
      const uint64_t dq0 = make_sdesc_sw128(smem_addr(s_q), 16, 1024);
      const uint32_t dp_lo = (uint32_t)dp0, dp_hi = (uint32_t)(dp0 >> 32);
      const uint32_t dq_lo = (uint32_t)dq0, dq_hi = (uint32_t)(dq0 >> 32);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < num_tiles; tile += tile_step) {
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          const uint32_t d = tmem_base + (uint32_t)(acc * BN);
          const uint32_t p_lo = dp_lo + (uint32_t)stage * (P_BYTES >> 4);
          const uint32_t q_lo = dq_lo + (uint32_t)stage * (cfg::Q_BYTES >> 4);
          if (elect_lane()) {
            // the accumulator is what is waited for: nothing but the MMAs comes after it
            ok = mbar_wait_short(&full[stage], phase, wb, SITE_E4M3_MMA) &&
                 mbar_wait_short(&acc_empty[acc], acc_phase ^ 1u, wb, SITE_E4M3_MMA);
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk) {
                if constexpr (PAIR)
                  mma_ss_f8_pair_w(d, p_lo + 2 * kk, dp_hi, q_lo + 2 * kk, dq_hi, idesc, kk != 0 ? 1u : 0u);
                else
                  mma_ss_f8_w(d, p_lo + 2 * kk, dp_hi, q_lo + 2 * kk, dq_hi, idesc, kk != 0 ? 1u : 0u);
              }
              if constexpr (PAIR) {
                mma_commit_pair(&acc_full[acc]);
                mma_commit_pair(&empty[stage]);
              } else {
                mma_commit(&acc_full[acc]);
                mma_commit(&empty[stage]);
              }
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      // Every MMA issued above completes before TMEM is released.
      if (elect_lane()) {
        if constexpr (PAIR) mma_commit_pair(drain);
        else mma_commit(drain);
      }
      __syncwarp();
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(drain, 0, wd, SITE_DRAIN);
    }
    if (warp >= 2) {
      // ------------------------------------------------------------ scales: P's by warp 2, Q's by warp 3
      const bool of_p = warp == 2;
      const int rows = of_p ? p.rows_p : p.rows_q;
      const long long ld = of_p ? p.ld_sp : p.ld_sq;
      const float* base = of_p ? p.sp : p.sq;
      const int shift = of_p ? p.p_shift : COLS ? 0 : 7;
      const int count = of_p ? BM : COLS ? BN : (BN + BM - 1) / BM;  // values of a block of K
      // four blocks by one load where they start on 16 bytes
      const bool vec = (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && (ld & 3) == 0 && (kb0 & 3) == 0;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < num_tiles; tile += tile_step) {
        int tp, tq;
        tile_coords(tile, num_p, num_q, p.group_p, tp, tq);
        const long long row0 = of_p ? (long long)tp * TILE_P + (PAIR ? rank * BM : 0) : (long long)tq * BN;
        for (int kb = kb0; kb < kb1; kb += KS) {
          ok = __all_sync(0xffffffffu, mbar_wait_short(&scale_empty[slot], phase ^ 1u, wb, SITE_E4M3_PRODUCER));
          if (!ok) break;
          float* to = s_scale + slot * cfg::SCALES + (of_p ? 0 : BM);
          // of four rows at once, so that eight loads are under way; pairs have few registers here, and wait
          // for something else
          constexpr int AT_ONCE = PAIR ? 1 : 4;
          for (int i0 = lane; i0 < count; i0 += 32 * AT_ONCE) {
            float4 v[AT_ONCE][KS / 4];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
              const int i = min(i0 + 32 * j, count - 1);
              const long long r = row0 + (of_p || COLS ? i : i * BM);
              const float* from = base + (min(r, (long long)rows - 1) >> shift) * ld + kb;
#pragma unroll
              for (int k = 0; k < KS; k += 4) {
                float4& x = v[j][k / 4];
                x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (vec && kb + k + 4 <= kb1) {
                  x = *reinterpret_cast<const float4*>(from + k);
                } else {
                  if (kb + k < kb1) x.x = from[k];
                  if (kb + k + 1 < kb1) x.y = from[k + 1];
                  if (kb + k + 2 < kb1) x.z = from[k + 2];
                  if (kb + k + 3 < kb1) x.w = from[k + 3];
                }
              }
            }
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
              const int i = i0 + 32 * j;
              if (i >= count) break;
#pragma unroll
              for (int k = 0; k < KS; k += 4) {
                to[k * (BM + QS) + i] = v[j][k / 4].x;
                to[(k + 1) * (BM + QS) + i] = v[j][k / 4].y;
                to[(k + 2) * (BM + QS) + i] = v[j][k / 4].z;
                to[(k + 3) * (BM + QS) + i] = v[j][k / 4].w;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&scale_full[slot]);
          slot ^= 1;
          if (slot == 0) phase ^= 1u;
        }
      }
    }
  } else {
    // -------------------------------------------------------------- sums
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quarter = warp & 3;         // TMEM lanes this warp may access
    const int half = (warp - 4) >> 2;     // of the tile's columns
    const int r_in_tile = quarter * 32 + lane;
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HALF);
    const uint32_t taken0 = cluster_addr(&acc_empty[0], 0), taken1 = cluster_addr(&acc_empty[1], 0);  // pairs
    int acc = 0, slot = 0;
    uint32_t acc_phase = 0, slot_phase = 0;
    // Every warp goes through every tile, and every lane through every block, also after a wait gave up: the warps
    // meet at barriers below, and the loads are the whole warp's, while each lane waits, and can give up, by
    // itself. It then waits and arrives no more; what it adds is of no use. (8192 x 8192 x 4096 with a scale per row of
    // both: 306 us, 311 with `ok` tested at each wait and arrival of a block, 314 with a vote of the warp there.)
    bool ok = true, arrives = lane == 0;
    auto waited = [&](bool done) {
      if (!done) ok = arrives = false;
    };
    for (int tile = first_tile; tile < num_tiles; tile += tile_step) {
      int tp, tq;
      tile_coords(tile, num_p, num_q, p.group_p, tp, tq);
      uint64_t sum[HALF / 2];
#pragma unroll
      for (int j = 0; j < HALF / 2; ++j) sum[j] = 0ull;
      // Shared memory is busy with the operands, and an access to it takes some 150 cycles: the scales of
      // a block's rows are read, and its product is first asked for, while the block before it is added.
      const float* scales = s_scale + slot * cfg::SCALES;
      bool ready;
      float f[QUAD ? 4 : 1];
      auto row_scales = [&]() {
        if constexpr (QUAD) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = scales[quarter * 32 + (lane >> 2) + 8 * e];
        } else {
          f[0] = scales[r_in_tile];
          if constexpr (!COLS) f[0] *= scales[BM + half];
        }
      };
      // the block is in registers, its scales too: on to the next
      auto taken = [&](int kb) {
        tc_fence_before();
        __syncwarp();
        if (arrives) {
          if constexpr (PAIR) mbar_arrive_cluster(acc ? taken1 : taken0);
          else mbar_arrive(&acc_empty[acc]);
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        const int done = kb + 1 - kb0;
        if (kb + 1 == kb1 || (done & (KS - 1)) == 0) {
          if (arrives) mbar_arrive(&scale_empty[slot]);
          slot ^= 1;
          if (slot == 0) slot_phase ^= 1u;
          scales = s_scale + slot * cfg::SCALES;
          if (ok && kb + 1 < kb1) waited(mbar_wait_short(&scale_full[slot], slot_phase, wb, SITE_E4M3_EPILOGUE));
        } else {
          scales += BM + QS;
        }
        if (kb + 1 < kb1) {
          ready = mbar_try_wait(&acc_full[acc], acc_phase) || !ok;
          row_scales();
        }
      };
      if (ok && kb0 < kb1) waited(mbar_wait_short(&scale_full[slot], slot_phase, wb, SITE_E4M3_EPILOGUE));
      ready = !ok;
      row_scales();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!ready) waited(mbar_wait_poll(&acc_full[acc], acc_phase, wb, SITE_E4M3_EPILOGUE));
        __syncwarp();
        tc_fence_after();
        const uint32_t from = lanes + (uint32_t)(acc * BN);
        const float* col_scales = scales + BM + half * HALF;
        // a load is under way while the columns of the one before it are added
        if constexpr (QUAD) {
          uint64_t rows[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) rows[e] = f2_pack(f[e], f[e]);
          uint32_t v[2][16];
          uint64_t cs[4];
          auto load = [&](int c, int hh) {
            tmem_ld_16x256(from + ((uint32_t)(16 * hh) << 16) + (uint32_t)c, v[hh]);
            if (hh == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 s = *reinterpret_cast<const float2*>(col_scales + c + 8 * i + 2 * (lane & 3));
                cs[i] = f2_pack(s.x, s.y);
              }
            }
          };
          load(0, 0);
#pragma unroll
          for (int c = 0; c < HALF; c += 32) {
            uint64_t now[4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              tmem_ld_wait16(v[hh]);
              if (hh == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = cs[i];
                load(c, 1);
              } else if (c + 32 < HALF) {
                load(c + 32, 0);
              } else {
                taken(kb);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  uint64_t& a = sum[((c >> 5) * 4 + 2 * hh + e) * 4 + i];
                  a = f2_fma(f2_pack(__uint_as_float(v[hh][4 * i + 2 * e]), __uint_as_float(v[hh][4 * i + 2 * e + 1])),
                             f2_mul(rows[2 * hh + e], now[i]), a);
                }
            }
          }
        } else {
          const uint64_t f2 = f2_pack(f[0], f[0]);
          uint32_t v[2][CH];
          float4 cs[2][COLS ? CH / 4 : 1];
          auto load = [&](int c) {
            tmem_ld<CH>(from + c, v[(c / CH) & 1]);
            if constexpr (COLS) {
#pragma unroll
              for (int j = 0; j < CH / 4; ++j) cs[(c / CH) & 1][j] = *reinterpret_cast<const float4*>(col_scales + c + 4 * j);
            }
          };
          load(0);
#pragma unroll
          for (int c = 0; c < HALF; c += CH) {
            uint32_t(&now)[CH] = v[(c / CH) & 1];
            tmem_wait<CH>(now);
            if (c + CH < HALF) load(c + CH);
            else taken(kb);
#pragma unroll
            for (int j = 0; j < CH; j += 2) {
              uint64_t scale = f2;
              if constexpr (COLS) {
                const float4& s = cs[(c / CH) & 1][j >> 2];
                scale = f2_mul(f2, (j & 2) ? f2_pack(s.z, s.w) : f2_pack(s.x, s.y));
              }
              uint64_t& a = sum[(c + j) >> 1];
              a = f2_fma(f2_pack(__uint_as_float(now[j]), __uint_as_float(now[j + 1])), scale, a);
            }
          }
        }
      }

      if constexpr (TURNED) {
        // this CTA's share of the sum, [column][row], where the ring was: every block has been taken
        float* part = reinterpret_cast<float*>(smem) + half * HALF * PART;
        if constexpr (QUAD) {
#pragma unroll
          for (int c = 0; c < HALF / 32; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float a, b;
                f2_unpack(sum[(c * 4 + e) * 4 + i], a, b);
                float* at = part + (32 * c + 8 * i + 2 * (lane & 3)) * PART + quarter * 32 + 8 * e + (lane >> 2);
                at[0] = a;
                at[PART] = b;
              }
        } else {
#pragma unroll
          for (int j = 0; j < HALF; j += 2) {
            float a, b;
            f2_unpack(sum[j >> 1], a, b);
            part[j * PART + r_in_tile] = a;
            part[(j + 1) * PART + r_in_tile] = b;
          }
        }
      } else {
        // through 32 KB of shared memory per warpgroup, as boxes of 128 rows x 128 bytes with their
        // 16-byte chunks swizzled by the row: two boxes of 64 bf16 columns, or in two rounds of 32 fp32
        uint8_t* out = s_out + half * 32768;
        const int warp_in = warp & 3;
        const bool leader = warp_in == 0 && lane == 0;
#pragma unroll
        for (int round = 0; round < 2; ++round) {
          if (round == 1 && !p.c_f32) break;
          if (leader) bulk_wait_read();  // the boxes are free
          asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
          if constexpr (QUAD) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 32 columns
              if (p.c_f32 && c >> 1 != round) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int r = quarter * 32 + 8 * e + (lane >> 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float a, b;
                  f2_unpack(sum[(c * 4 + e) * 4 + i], a, b);
                  if (p.c_f32)
                    *reinterpret_cast<float2*>(out + (c & 1) * 16384 + r * 128 +
                                               (((2 * i + ((lane & 3) >> 1)) ^ (r & 7)) << 4) + (lane & 1) * 8) =
                        make_float2(a, b);
                  else
                    *reinterpret_cast<uint32_t*>(out + (c >> 1) * 16384 + r * 128 +
                                                 ((((c & 1) * 4 + i) ^ (r & 7)) << 4) + (lane & 3) * 4) = pack_bf16x2(a, b);
                }
              }
            }
          } else if (p.c_f32) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // 16 chunks of 4 columns
              float a, b, c, d;
              f2_unpack(sum[32 * round + 2 * j], a, b);
              f2_unpack(sum[32 * round + 2 * j + 1], c, d);
              *reinterpret_cast<float4*>(out + (j >> 3) * 16384 + r_in_tile * 128 + (((j & 7) ^ (r_in_tile & 7)) << 4)) =
                  make_float4(a, b, c, d);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // 16 chunks of 8 columns
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float a, b;
                f2_unpack(sum[4 * j + e], a, b);
                w[e] = pack_bf16x2(a, b);
              }
              *reinterpret_cast<uint4*>(out + (j >> 3) * 16384 + r_in_tile * 128 + (((j & 7) ^ (r_in_tile & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async();
          asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
          const int first_col = tq * BN + half * HALF + round * 64;
          const int first_row = tp * TILE_P + (PAIR ? rank * BM : 0);
          if (p.tma_out) {
            if (leader) {
              const int per = p.c_f32 ? 32 : 64;
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (first_col + b * per < p.rows_q && first_row < p.rows_p)
                  tma_store_2d(&tm_c, out + b * 16384, first_col + b * per, first_row);
              bulk_commit();
            }
          } else {
            // row by row, a column per lane
            const int columns = p.rows_q - first_col, rows = p.rows_p - (first_row + warp_in * 32);
            const long long at = (long long)(first_row + warp_in * 32) * p.ldc + first_col + lane;
            const uint8_t* from = out + warp_in * 32 * 128;
            if (p.c_f32) {
              float* to = static_cast<float*>(p.c) + at;
#pragma unroll 8
              for (int i = 0; i < 32; ++i) {
                if (i >= rows) break;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  if (lane + 32 * b >= columns) continue;
                  const float x = *reinterpret_cast<const float*>(from + b * 16384 + i * 128 +
                                                                  (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
                  float* c = to + i * p.ldc + 32 * b;
                  *c = p.accumulate ? *c + x : x;
                }
              }
            } else {
              __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.c) + at;
#pragma unroll 8
              for (int i = 0; i < 32; ++i) {
                if (i >= rows) break;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  if (lane + 32 * b >= columns) continue;
                  to[i * p.ldc + 32 * b] = *reinterpret_cast<const __nv_bfloat16*>(
                      from + (b >> 1) * 16384 + i * 128 + (((4 * (b & 1) + (lane >> 3)) ^ (i & 7)) << 4) + (lane & 7) * 2);
                }
              }
            }
          }
        }
      }
    }
    if constexpr (!TURNED) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster.sync();  // neither leaves while the other may reach its memory
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, cfg::TMEM_COLS);
    else tmem_dealloc(tmem_base, cfg::TMEM_COLS);
  }
  if constexpr (TURNED) {
    // each CTA of the cluster joins and writes some of the columns
    if (split > 1) cluster.sync();
    int tp, tq;
    tile_coords(first_tile, num_p, num_q, p.group_p, tp, tq);
    const int cols = min(BN, p.rows_q - tq * BN);
    const int c0 = cols * rank / split, c1 = cols * (rank + 1) / split;
    for (int i = c0 * BM + threadIdx.x; i < c1 * BM; i += THREADS) {
      const long long row = (long long)tp * BM + (i & (BM - 1));
      if (row >= p.rows_p) continue;
      const float* mine = reinterpret_cast<const float*>(smem) + (i >> 7) * PART + (i & (BM - 1));
      float v = 0.f;
      if (split == 1) v = *mine;
      else
        for (int s = 0; s < split; ++s) v += *cluster.map_shared_rank(mine, s);
      put(p, (long long)(tq * BN + (i >> 7)) * p.ldc + row, v);
    }
    if (split > 1) cluster.sync();  // the others have read this CTA's share
  }
}

template <int BN, bool COLS, bool TURNED, bool PAIR>
tsp_status launch(const CUtensorMap& tp, const CUtensorMap& tq, const CUtensorMap& tc, const Params& p, int ctas, int cluster, cudaStream_t s) {
  auto kernel = matmul_e4m3_kernel<BN, COLS, TURNED, PAIR>;
  constexpr size_t smem = Config<BN, COLS, PAIR>::SMEM_BYTES;
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem, "matmul_e4m3: cudaFuncSetAttribute"));
  const cudaError_t e = launch_early_cluster(kernel, ctas, THREADS, smem, s, cluster, tp, tq, tc, p);
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "matmul_e4m3: launch");
}

struct Operand {
  const uint8_t* x;
  int64_t rows, ld;
  const float* scales;
  int64_t ld_scales;
  int shift;  // 0: a scale for every row, 7: one for 128 rows
};

// split: CTAs on the blocks of K of one tile; a pair takes the whole of K.
template <int BN, bool COLS, bool TURNED, bool PAIR>
tsp_status run(const Operand& op, const Operand& oq, int64_t k, Params p, int split, cudaStream_t s) {
  CUtensorMap tp, tq, tc{};
  TSP_TRY(make_tmap_2d_u8(&tp, op.x, (uint64_t)k, (uint64_t)op.rows, (uint64_t)op.ld, BK, BM));
  TSP_TRY(make_tmap_2d_u8(&tq, oq.x, (uint64_t)k, (uint64_t)oq.rows, (uint64_t)oq.ld, BK, PAIR ? BN / 2 : BN));
  if (!TURNED && p.tma_out) {
    if (p.c_f32)
      TSP_TRY(make_tmap_2d_f32(&tc, p.c, (uint64_t)oq.rows, (uint64_t)op.rows, (uint64_t)p.ldc * 4, 32, BM));
    else
      TSP_TRY(make_tmap_2d_bf16(&tc, p.c, (uint64_t)oq.rows, (uint64_t)op.rows, (uint64_t)p.ldc * 2, 64, BM));
  }
  p.rows_p = (int)op.rows;
  p.rows_q = (int)oq.rows;
  p.sp = op.scales;
  p.ld_sp = op.ld_scales;
  p.p_shift = op.shift;
  p.sq = oq.scales;
  p.ld_sq = oq.ld_scales;
  constexpr int tile_p = PAIR ? 2 * BM : BM;
  const int cluster = PAIR ? 2 : split;
  const int64_t tiles = ((op.rows + tile_p - 1) / tile_p) * ((oq.rows + BN - 1) / BN);
  if (tiles * cluster > (1ll << 30)) return fail(TSP_ERR_UNSUPPORTED, "tsp_matmul_e4m3: too many tiles");
  const int64_t clusters = TURNED ? tiles : std::min<int64_t>(tiles, std::max(1, sm_count() / cluster));
  return launch<BN, COLS, TURNED, PAIR>(tp, tq, tc, p, (int)(clusters * cluster), cluster, s);
}

}  // namespace
}  // namespace tsp

using namespace tsp;

extern "C" {

size_t tsp_matmul_e4m3_workspace_bytes(void) { return 256; }

tsp_status tsp_matmul_e4m3(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t ld_a, const float* a_scales,
                           const uint8_t* b, int64_t ld_b, const float* b_scales, int b_block, void* c, int64_t ld_c,
                           int c_f32, int accumulate, void* ws, void* stream) {
  TSP_GUARD_BEGIN
  const std::string w("tsp_matmul_e4m3");
  constexpr int64_t most = 1ll << 30;
  if (m < 0 || n < 0 || k < 0 || m > most || n > most || k > most)
    return fail(TSP_ERR_UNSUPPORTED, w + ": m, n and k in [0, 2^30]");
  if (b_block != 1 && b_block != 128) return fail(TSP_ERR_UNSUPPORTED, w + ": b_block 1 or 128");
  if (accumulate && !c_f32) return fail(TSP_ERR_UNSUPPORTED, w + ": only an fp32 output can be added to");
  if (m == 0 || n == 0) return TSP_OK;
  if (!c) return fail(TSP_ERR_INVALID_ARG, w + ": null pointer");
  const unsigned es = c_f32 ? 4u : 2u;
  if (reinterpret_cast<uintptr_t>(c) % es) return fail(TSP_ERR_INVALID_ARG, w + ": c not aligned to its element");
  if (ld_c < n || ld_c > (1ll << 40)) return fail(TSP_ERR_INVALID_ARG, w + ": row stride of c");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (k == 0) {  // an empty sum
    if (accumulate) return TSP_OK;
    const cudaError_t e = cudaMemset2DAsync(c, (size_t)ld_c * es, 0, (size_t)n * es, (size_t)m, s);
    return e == cudaSuccess ? TSP_OK : cuda_fail(e, "tsp_matmul_e4m3: memset");
  }
  TSP_TRY(check_ws(ws, "tsp_matmul_e4m3"));
  if (!a || !b || !a_scales || !b_scales) return fail(TSP_ERR_INVALID_ARG, w + ": null pointer");
  if (!al16(a) || !al16(b) || ld_a % 16 || ld_b % 16)
    return fail(TSP_ERR_INVALID_ARG, w + ": rows of a and b must start on 16 bytes");
  if (ld_a < k || ld_b < k || ld_a > (1ll << 39) || ld_b > (1ll << 39))
    return fail(TSP_ERR_INVALID_ARG, w + ": row stride of a or b");
  if (reinterpret_cast<uintptr_t>(a_scales) % 4 || reinterpret_cast<uintptr_t>(b_scales) % 4)
    return fail(TSP_ERR_INVALID_ARG, w + ": scales not aligned to their element");
  const int64_t nkb = (k + BK - 1) / BK;
  const int64_t sa = m * nkb * 4, sb = (b_block == 1 ? n : (n + 127) / 128) * nkb * 4;
  const Extent out = extent(c, m, n * es, ld_c * es);
  for (const Extent& in : {extent(a, m, k, ld_a), extent(b, n, k, ld_b), extent(a_scales, 1, sa, sa), extent(b_scales, 1, sb, sb)})
    if (overlaps(out, in)) return fail(TSP_ERR_INVALID_ARG, w + ": c aliases an input");
  const Operand oa{a, m, ld_a, a_scales, nkb, 0};
  const Operand ob{b, n, ld_b, b_scales, nkb, b_block == 1 ? 0 : 7};
  Params p{};
  p.nkb = (int)nkb;
  p.c = c;
  p.ldc = ld_c;
  p.c_f32 = c_f32;
  p.accumulate = accumulate;
  // TMA writes whole 16 bytes: a row that ends inside them would take what lies behind it along
  p.tma_out = !accumulate && al16(c) && (ld_c * es) % 16 == 0 && (n * es) % 16 == 0;
  p.group_p = 1;
  p.status = status_of(ws);
  p.limit_ns = wait_limit_ns();

  // Which kernel, by estimates in tenths of a microsecond of what each takes: so many per block of K and wave of
  // CTAs, and so many around. Measured on both sides (us, pairs / turned): 512 x 4096 x 4096 19.7 / 21.3,
  // 256 x 4096 x 4096 19.4 / 18.1, 2048^3 13.8 / 28.4, 1024 x 1024 x 8192 with a scale per row of both 46.9 / 24.6,
  // 256 x 256 x 8192 43 / 10, 2816 x 1024 x 1000 14.5 / 21.4. Up to 128 rows a pair's tile would be half empty.
  const int64_t sms = sm_count();
  const int bn = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const int64_t tiles = ((n + BM - 1) / BM) * ((m + bn - 1) / bn);
  const int64_t slots = (bn <= 32 ? 2 : 1) * sms;
  int split = 1;  // as many CTAs as there is room for at once (more waves: 48 x 11008 x 4096 17 -> 23 us)
  while (split < 8 && tiles * (split + 1) <= slots && nkb >= (split + 1) * 2) ++split;
  const int64_t turned = (tiles * split + slots - 1) / slots * (6 * ((nkb + split - 1) / split) + 10) + (split > 1 ? 60 : 40);
  const int64_t pair_tiles = ((m + 255) / 256) * ((n + 255) / 256);
  const int64_t pairs = (pair_tiles + sms / 2 - 1) / std::max<int64_t>(1, sms / 2) * ((b_block == 1 ? 13 : 9) * nkb / 2 + 10) + 40;
  if (m > 128 && pairs <= turned) {
    p.group_p = walk_group(m, n, k, 2 * BM);
    return b_block == 1 ? run<256, true, false, true>(oa, ob, k, p, 1, s) : run<256, false, false, true>(oa, ob, k, p, 1, s);
  }
  switch (bn) {
    case 16: return run<16, true, true, false>(ob, oa, k, p, split, s);
    case 32: return run<32, true, true, false>(ob, oa, k, p, split, s);
    case 64: return run<64, true, true, false>(ob, oa, k, p, split, s);
    default: return run<128, true, true, false>(ob, oa, k, p, split, s);
  }
  TSP_GUARD_END
}

}  // extern "C"
