// matmul_e4m3.cu - the product of two e4m3 matrices with fp32 scales for blocks of 128:
//     C[m][n] = sum over blocks kb of K  sa[m][kb] sb[n][kb]  sum over k in kb  a[m][k] b[n][k]
// both operands K-major, the inner sum on the tensor cores (tcgen05, kind::f8f6f4), the outer one in
// fp32 registers: the scales are arbitrary fp32 numbers, so a block's product has to leave tensor
// memory before it can be scaled and added.
//
// One CTA holds a tile of 128 rows of one operand (P, the lanes of tensor memory) and BN rows of the other
// (Q, its columns), 384 threads:
//   warp 0      TMA producer: 128-byte K blocks of P and Q into a ring of 128B-swizzled buffers
//   warp 1      one lane issues the block's four MMAs (M = 128, N = BN, K = 32) into one of two
//               accumulators in tensor memory, each block from zero
//   warps 4..11 take a finished accumulator (a row and BN / 2 columns per thread), scale it and add
//               it to the tile's sum in registers, while the next block's MMAs run
// Large products: P = A, Q = B with BN = 256, persistent CTAs. Few rows or few tiles: P = B, Q = A
// with BN >= the rows of A, and the blocks of K split over a cluster of CTAs, which join their sums through
// distributed shared memory in a fixed order.
#include <cooperative_groups.h>

#include <algorithm>

#include "tsp_device.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr uint32_t P_BYTES = BM * BK;

template <int BN>
struct Config {
  static constexpr uint32_t Q_BYTES = BN * BK;
  static constexpr uint32_t STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr uint32_t TMEM_COLS = BN < 16 ? 32 : 2 * BN;
  static constexpr int CH = BN >= 64 ? 32 : BN / 2;  // columns per tensor memory load
  static constexpr size_t SCALE_BYTES = 2 * BN * 4;
  static constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * STAGE_BYTES + SCALE_BYTES + 256;
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
  int wide;     // C's rows start on 32 bytes
  int group_p;  // tile order of the persistent walk
  DevStatus* status;
  unsigned long long limit_ns;
};

__device__ __forceinline__ void tile_coords(int tile, int num_p, int num_q, int group_p, int& tp, int& tq) {
  const int span = group_p * num_q;
  const int g = tile / span, r = tile - g * span;
  const int first = g * group_p;
  const int gm = min(group_p, num_p - first);
  tp = first + r % gm;
  tq = r / gm;
}

template <int CH>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[CH]) {
  if constexpr (CH == 32) tmem_ld32(addr, r);
  else if constexpr (CH == 16) tmem_ld16(addr, r);
  else tmem_ld8(addr, r);
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(EPI_THREADS) : "memory"); }

__device__ __forceinline__ void put(const Params& p, long long at, float v) {
  if (p.c_f32) {
    float* c = static_cast<float*>(p.c) + at;
    *c = p.accumulate ? *c + v : v;
  } else {
    static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
  }
}

__device__ __forceinline__ void st_v8(void* ptr, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// COLS: Q has a scale for every row (a column of the tile), else one for 128 rows.
// TURNED: P = B and Q = A, C[q][p]; else C[p][q].
template <int BN, bool COLS, bool TURNED>
__global__ void __launch_bounds__(THREADS, 1)
    matmul_e4m3_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                       const Params p) {
  using cfg = Config<BN>;
  constexpr int STAGES = cfg::STAGES, CH = cfg::CH, HALF = BN / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* s_p = smem;
  uint8_t* s_q = smem + STAGES * P_BYTES;
  float* s_scale = reinterpret_cast<float*>(smem + STAGES * cfg::STAGE_BYTES);  // [2][BN]
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_scale) + cfg::SCALE_BYTES);
  uint64_t* full = bars;                   // [STAGES] TMA landed
  uint64_t* empty = bars + STAGES;         // [STAGES] MMAs reading the stage are done
  uint64_t* acc_full = bars + 2 * STAGES;  // [2] a block's product is complete
  uint64_t* acc_empty = acc_full + 2;      // [2] it has been taken
  uint64_t* drain = acc_empty + 2;         // [1] every MMA issued has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.num_blocks();
  const int rank = (int)cluster.block_rank();

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_p = (p.rows_p + BM - 1) / BM;
  const int num_q = (p.rows_q + BN - 1) / BN;
  const int num_tiles = num_p * num_q;
  const int first_tile = blockIdx.x / split, tile_step = gridDim.x / split;
  const int kb0 = (int)((long long)p.nkb * rank / split), kb1 = (int)((long long)p.nkb * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_p);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, cfg::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  dependents_may_start();
  prior_kernel_done();

  WaitBound wb{p.status, p.limit_ns, abort_flag};

  // Registers: 384 threads start with 168 each, the most that three warps per scheduler leave; the
  // sums of a wide tile (128 of them per thread) need more. 4 x 72 + 8 x 216 = 12 x 168.
  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
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
          if (!mbar_wait(&empty[stage], phase ^ 1u, wb, SITE_E4M3_PRODUCER)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], cfg::STAGE_BYTES);
          tma_load_2d(s_p + stage * P_BYTES, &tm_p, &full[stage], kb * BK, tp * BM);
          tma_load_2d(s_q + stage * cfg::Q_BYTES, &tm_q, &full[stage], kb * BK, tq * BN);
#pragma unroll
          for (int s = 0; s < STAGES; ++s)
            if (s == stage) last_parity[s] = (int)phase;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Do not leave while a TMA copy into this CTA's shared memory is in flight.
      WaitBound wd{p.status, p.limit_ns, nullptr};
#pragma unroll
      for (int s = 0; s < STAGES; ++s)
        if (last_parity[s] >= 0) mbar_wait(&full[s], (uint32_t)last_parity[s], wd, SITE_DRAIN);
    }
    if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = make_idesc_e4m3(BM, BN);
      const uint64_t dp0 = make_sdesc_sw128(smem_addr(s_p), 16, 1024);
      const uint64_t dq0 = make_sdesc_sw128(smem_addr(s_q), 16, 1024);
      const uint32_t dp_lo = (uint32_t)dp0, dp_hi = (uint32_t)(dp0 >> 32);
      const uint32_t dq_lo = (uint32_t)dq0, dq_hi = (uint32_t)(dq0 >> 32);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < num_tiles; tile += tile_step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, wb, SITE_E4M3_MMA) ||
              !mbar_wait(&full[stage], phase, wb, SITE_E4M3_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * BN);
          const uint32_t p_lo = dp_lo + (uint32_t)stage * (P_BYTES >> 4);
          const uint32_t q_lo = dq_lo + (uint32_t)stage * (cfg::Q_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_ss_f8_w(d, p_lo + 2 * kk, dp_hi, q_lo + 2 * kk, dq_hi, idesc, kk != 0 ? 1u : 0u);
          mma_commit(&empty[stage]);
          mma_commit(&acc_full[acc]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      // Every MMA issued above completes before TMEM is released.
      mma_commit(drain);
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(drain, 0, wd, SITE_DRAIN);
    }
  } else {
    // -------------------------------------------------------------- sums
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp & 3;         // TMEM lanes this warp may access
    const int half = (warp - 4) >> 2;     // of the tile's columns
    const int r_in_tile = quarter * 32 + lane;
    const int tid = threadIdx.x - 128;
    const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HALF);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int tile = first_tile; tile < num_tiles; tile += tile_step) {
      int tp, tq;
      tile_coords(tile, num_p, num_q, p.group_p, tp, tq);
      uint64_t sum[HALF / 2];
#pragma unroll
      for (int j = 0; j < HALF / 2; ++j) sum[j] = 0ull;
      const long long row = (long long)tp * BM + r_in_tile;
      const float* row_scale = p.sp + (min(row, (long long)p.rows_p - 1) >> p.p_shift) * p.ld_sp;
      // the scale of a column per thread, or that of this half's block
      const long long col = (long long)tq * BN + (COLS ? tid : half * HALF);
      const float* col_scale = p.sq + (min(col, (long long)p.rows_q - 1) >> (COLS ? 0 : 7)) * p.ld_sq;
      const bool loads = !COLS || tid < BN;
      // one block ahead (two for what goes through shared memory)
      float rs = kb0 < kb1 ? row_scale[kb0] : 0.f;
      float cs = 0.f;
      if (loads && kb0 < kb1) cs = col_scale[kb0];
      if constexpr (COLS) {
        epilogue_sync();  // the last tile's scales have been read
        if (loads) {
          s_scale[(kb0 & 1) * BN + tid] = cs;
          if (kb0 + 1 < kb1) cs = col_scale[kb0 + 1];
        }
      }
      for (int kb = kb0; kb < kb1; ++kb) {
        const float rs_now = rs, cs_now = cs;
        if (kb + 1 < kb1) rs = row_scale[kb + 1];
        if constexpr (COLS) {
          epilogue_sync();
          if (loads && kb + 1 < kb1) {
            s_scale[((kb + 1) & 1) * BN + tid] = cs;
            if (kb + 2 < kb1) cs = col_scale[kb + 2];
          }
        } else {
          if (kb + 1 < kb1) cs = col_scale[kb + 1];
        }
        ok = ok && mbar_wait(&acc_full[acc], acc_phase, wb, SITE_E4M3_EPILOGUE);
        if (ok) {
          tc_fence_after();
          const uint32_t from = lanes + (uint32_t)(acc * BN);
          const float f = COLS ? rs_now : rs_now * cs_now;
          const uint64_t f2 = f2_pack(f, f);
#pragma unroll
          for (int c = 0; c < HALF; c += CH) {
            uint32_t v[CH];
            tmem_ld<CH>(from + c, v);
            tmem_ld_wait();
            if constexpr (COLS) {
              const float4* s4 = reinterpret_cast<const float4*>(s_scale + (kb & 1) * BN + half * HALF + c);
#pragma unroll
              for (int j = 0; j < CH; j += 4) {
                const float4 s = s4[j >> 2];
                uint64_t& a = sum[(c + j) >> 1];
                uint64_t& b = sum[((c + j) >> 1) + 1];
                a = f2_fma(f2_pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2_mul(f2, f2_pack(s.x, s.y)), a);
                b = f2_fma(f2_pack(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), f2_mul(f2, f2_pack(s.z, s.w)), b);
              }
            } else {
#pragma unroll
              for (int j = 0; j < CH; j += 2) {
                uint64_t& a = sum[(c + j) >> 1];
                a = f2_fma(f2_pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2, a);
              }
            }
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }

      if (split > 1) {
        // this CTA's share of the sum, [column][row]; the ring is idle: every block has been taken
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int j = 0; j < HALF; j += 2) {
          float a, b;
          f2_unpack(sum[j >> 1], a, b);
          part[(half * HALF + j) * BM + r_in_tile] = a;
          part[(half * HALF + j + 1) * BM + r_in_tile] = b;
        }
        continue;  // one tile per cluster
      }
      const bool row_ok = row < p.rows_p;
      const long long q0 = (long long)tq * BN + half * HALF;
      if (!row_ok) continue;
      if constexpr (TURNED) {
#pragma unroll
        for (int j = 0; j < HALF; j += 2) {
          float a, b;
          f2_unpack(sum[j >> 1], a, b);
          if (q0 + j < p.rows_q) put(p, (q0 + j) * p.ldc + row, a);
          if (q0 + j + 1 < p.rows_q) put(p, (q0 + j + 1) * p.ldc + row, b);
        }
      } else if (p.wide && q0 + HALF <= p.rows_q) {
        if (p.c_f32) {
          float* c = static_cast<float*>(p.c) + row * p.ldc + q0;
#pragma unroll
          for (int j = 0; j < HALF; j += 8) {
            float f[8];
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) f2_unpack(sum[(j + e) >> 1], f[e], f[e + 1]);
            if (p.accumulate) {
              const float4 x = *reinterpret_cast<const float4*>(c + j), y = *reinterpret_cast<const float4*>(c + j + 4);
              f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w, f[4] += y.x, f[5] += y.y, f[6] += y.z, f[7] += y.w;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(f[e]);
            st_v8(c + j, w);
          }
        } else {
          __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.c) + row * p.ldc + q0;
#pragma unroll
          for (int j = 0; j < HALF; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float a, b;
              f2_unpack(sum[(j >> 1) + e], a, b);
              w[e] = pack_bf16x2(a, b);
            }
            st_v8(c + j, w);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < HALF; j += 2) {
          float a, b;
          f2_unpack(sum[j >> 1], a, b);
          if (q0 + j < p.rows_q) put(p, row * p.ldc + q0 + j, a);
          if (q0 + j + 1 < p.rows_q) put(p, row * p.ldc + q0 + j + 1, b);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, cfg::TMEM_COLS);
  }
  if constexpr (TURNED) {
    if (split > 1) {
      cluster.sync();
      int tp, tq;
      tile_coords(first_tile, num_p, num_q, p.group_p, tp, tq);
      const float* mine = reinterpret_cast<const float*>(smem);
      const int c0 = BN * rank / split, c1 = BN * (rank + 1) / split;
      for (int i = c0 * BM + threadIdx.x; i < c1 * BM; i += THREADS) {
        float v = 0.f;
        for (int s = 0; s < split; ++s) v += *cluster.map_shared_rank(mine + i, s);
        const long long row = (long long)tp * BM + (i & (BM - 1)), col = (long long)tq * BN + (i >> 7);
        if (row < p.rows_p && col < p.rows_q) put(p, col * p.ldc + row, v);
      }
      cluster.sync();  // the others have read this CTA's share
    }
  }
}

template <int BN, bool COLS, bool TURNED>
tsp_status launch(const CUtensorMap& tp, const CUtensorMap& tq, const Params& p, int ctas, int split, cudaStream_t s) {
  auto kernel = matmul_e4m3_kernel<BN, COLS, TURNED>;
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)Config<BN>::SMEM_BYTES,
                            "matmul_e4m3: cudaFuncSetAttribute"));
  const cudaError_t e = launch_early_cluster(kernel, ctas, THREADS, Config<BN>::SMEM_BYTES, s, split, tp, tq, p);
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "matmul_e4m3: launch");
}

struct Operand {
  const uint8_t* x;
  int64_t rows, ld;
  const float* scales;
  int64_t ld_scales;
  int shift;  // 0: a scale for every row, 7: one for 128 rows
};

template <int BN, bool COLS, bool TURNED>
tsp_status run(const Operand& op, const Operand& oq, int64_t k, Params p, int split, cudaStream_t s) {
  CUtensorMap tp, tq;
  TSP_TRY(make_tmap_2d_u8(&tp, op.x, (uint64_t)k, (uint64_t)op.rows, (uint64_t)op.ld, BK, BM));
  TSP_TRY(make_tmap_2d_u8(&tq, oq.x, (uint64_t)k, (uint64_t)oq.rows, (uint64_t)oq.ld, BK, BN));
  p.rows_p = (int)op.rows;
  p.rows_q = (int)oq.rows;
  p.sp = op.scales;
  p.ld_sp = op.ld_scales;
  p.p_shift = op.shift;
  p.sq = oq.scales;
  p.ld_sq = oq.ld_scales;
  const int64_t tiles = ((op.rows + BM - 1) / BM) * ((oq.rows + BN - 1) / BN);
  if (tiles * split > (1ll << 30)) return fail(TSP_ERR_UNSUPPORTED, "tsp_matmul_e4m3: too many tiles");
  const int64_t ctas = split > 1 ? tiles * split : std::min<int64_t>(tiles, sm_count());
  return launch<BN, COLS, TURNED>(tp, tq, p, (int)ctas, split, s);
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
  if (c == static_cast<const void*>(a) || c == static_cast<const void*>(b) || c == static_cast<const void*>(a_scales) ||
      c == static_cast<const void*>(b_scales))
    return fail(TSP_ERR_INVALID_ARG, w + ": c aliases an input");
  const int64_t nkb = (k + BK - 1) / BK;
  const Operand oa{a, m, ld_a, a_scales, nkb, 0};
  const Operand ob{b, n, ld_b, b_scales, nkb, b_block == 1 ? 0 : 7};
  Params p{};
  p.nkb = (int)nkb;
  p.c = c;
  p.ldc = ld_c;
  p.c_f32 = c_f32;
  p.accumulate = accumulate;
  p.wide = (reinterpret_cast<uintptr_t>(c) & 31u) == 0 && (ld_c * es) % 32 == 0;
  p.group_p = 1;
  p.status = status_of(ws);
  p.limit_ns = wait_limit_ns();

  const int64_t large = ((m + BM - 1) / BM) * ((n + 255) / 256);
  if (m > 128 && large >= sm_count() / 2) {
    // about 32 MB of A's row blocks walk down each column block of B together where B does not fit the L2 well
    const int64_t g = n * k <= (48ll << 20) ? 1 : (32ll << 20) / (BM * k);
    p.group_p = (int)std::max<int64_t>(1, g);
    return b_block == 1 ? run<256, true, false>(oa, ob, k, p, 1, s) : run<256, false, false>(oa, ob, k, p, 1, s);
  }
  const int bn = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const int64_t tiles = ((n + BM - 1) / BM) * ((m + bn - 1) / bn);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 2 * sm_count() && nkb >= split * 4) split *= 2;
  switch (bn) {
    case 16: return run<16, true, true>(ob, oa, k, p, split, s);
    case 32: return run<32, true, true>(ob, oa, k, p, split, s);
    case 64: return run<64, true, true>(ob, oa, k, p, split, s);
    default: return run<128, true, true>(ob, oa, k, p, split, s);
  }
  TSP_GUARD_END
}

}  // extern "C"
