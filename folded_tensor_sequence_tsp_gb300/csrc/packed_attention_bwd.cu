// packed_attention_bwd.cu - backward of the packed attention with grouped heads.
//
// With s_ij = q_i.k_j over the pairs of one sequence with j <= i, P_ij = exp2(s_ij
// scale_log2 - lse_i), dP_ij = dO_i.v_j and Delta_i = dO_i.o_i:
//     dS_ij = P_ij (dP_ij - Delta_i)
//     dQ_i = scale sum_j dS_ij k_j
//     dV_j = sum_i P_ij dO_i,   dK_j = scale sum_i dS_ij q_i,   i over the whole head group
// Bound: the tensor cores. Five products per visible pair are the gradient's own; the two
// kernels below both form S and dP, so seven run.
//
//   query side (first): a CTA owns one query tile (TPT tokens x G heads, 128 rows) and
//             streams the key tiles it sees: S = Q K^T, dP = dO V^T, dQ += dS K, with Q and
//             dO in TMEM as A operands. It also forms Delta, from its rows of o and dO, or
//             from P and dP where one key tile holds all keys of its rows, and leaves it for
//             the key side.
//   key side  a CTA owns 128 keys of one key head and streams every query tile that sees
//             them: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q. A tile's rows
//             are all heads of the group, so the group's sum needs nothing more: it happens
//             in the fp32 accumulators, in a fixed order.
// P and dS are rounded to bf16 as operands of the tensor core, 2^-9 relative per term; dS is
// formed from the unrounded P. Accumulators and statistics are fp32.
//
// Rows that are no query of the sequence (the rows of a tile behind the sequence's end, and
// those past TPT x G when G does not divide 128) enter the key side's sums with P = 0: their
// lse is +infinity and their Q and dO rows are zeros in shared memory, so nothing that lies
// behind the sequence can reach a sum. The query side clears its last K and V tile the same
// way. Pairs above the diagonal are set to 0 by selection, in P and in dS.
//
// Schedules (per streamed tile j; products of one issuing lane execute in order): query side
// S(j+1), dQ(j), dP(j+1); key side dV(j), S^T(j+1), dK(j), dP^T(j+1) with two 128-column
// regions that swap roles from tile to tile. The element-wise warps' exponentials and
// products run under the other product of their tile.
// TMEM columns, key side: dV [0, d), dK [d, 2d), regions [256, 384) and [384, 512).
// Query side: dQ [0, d), bf16 Q [d, 3d/2), bf16 dO [3d/2, 2d), S [256, 384), dP [384, 512).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attention_math.cuh"
#include "packed_attention.cuh"

namespace tsp {
namespace packed {
namespace {

constexpr int GCOLS = 64;  // streamed-tile columns per element-wise warpgroup
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_SC = 256, TM_DP = 384;  // query side
__device__ __forceinline__ uint32_t tm_s(int j) { return (j & 1) ? 384u : 256u; }
__device__ __forceinline__ uint32_t tm_g(int j) { return (j & 1) ? 256u : 384u; }

struct BwdParams {
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  long long ld_dq, ld_dk, ld_dv;
  const __nv_bfloat16* q;
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  long long ld_q, ld_o, ld_do;
  const float* lse;
  long long ld_lse;
  float* delta;
  long long ld_delta;
  Source src;
  int G, TPT, RU;
  float scale_log2, scale;
  DevStatus* status;
  unsigned long long limit_ns;
};

template <int HD>
struct KeyGeom {
  static constexpr int THREADS = 352;  // TMA, MMA, 2 x 4 element-wise warps, statistics
  static constexpr int BOXES = HD / 64;
  static constexpr uint32_t TILE_B = 128 * HD * 2;
  // Q tiles (with lse) and dO tiles (with Delta) in separate rings: a Q tile is read last
  // by dK, a full tile after its scores, so it gets the deeper ring
  static constexpr int QS = 3;
  static constexpr int OS = 2;
  static constexpr uint32_t SMALL = (QS + OS) * 512 + 256;
  static constexpr uint32_t TILES_OFF = (SMALL + 1023) / 1024 * 1024;
  static constexpr size_t USED = TILES_OFF + (size_t)(2 + QS + OS) * TILE_B;
  static constexpr size_t SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
};
static_assert(KeyGeom<128>::USED <= 227 * 1024, "key-side shared memory");

template <int HD>
struct QueryGeom {
  static constexpr int THREADS = 320;
  static constexpr int BOXES = HD / 64;
  static constexpr uint32_t TILE_B = 128 * HD * 2;
  static constexpr int KV_STAGES = 3;
  static constexpr uint32_t STAGE = 2 * TILE_B;  // K, V
  static constexpr size_t USED = 1024 + KV_STAGES * (size_t)STAGE + 1280;
  static constexpr size_t SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr uint32_t TM_Q = HD;
  static constexpr uint32_t TM_DO = HD + HD / 2;
};

// K-major operand offset (>> 4) of the kk-th 16-wide K step of a [rows][HD] tile stored as
// 64-column boxes.
__device__ __forceinline__ uint32_t kmajor_step(int kk) {
  return (uint32_t)(((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4);
}

// TMEM column of the bf16 A operand for the kk-th 16-wide step of a streamed tile's 128
// columns: warpgroup g's 64 values sit in the first 32 columns of its 64-column block.
__device__ __forceinline__ uint32_t packed_step(uint32_t base, int kk) {
  return base + (uint32_t)((kk >> 2) * GCOLS + (kk & 3) * 8);
}

// Zeros in the rows [from, 128) of a tile of `boxes` boxes, by `lanes` threads.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int boxes, int from, int lane, int lanes) {
  for (int b = 0; b < boxes; ++b) {
    uint4* rows = reinterpret_cast<uint4*>(tile + b * BOX_BYTES);
    for (int i = from * 8 + lane; i < 128 * 8; i += lanes) rows[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ============================================================== key side
template <int HD>
__global__ void __launch_bounds__(KeyGeom<HD>::THREADS, 1)
    packed_bwd_dkv_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmDO,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const BwdParams p) {
  using Geo = KeyGeom<HD>;
  Item it;
  {
    const int per_group = p.src.max_items * p.src.group;
    const int grp = (int)blockIdx.x / per_group;
    if (!find_item(p.src, grp, (int)blockIdx.x - grp * per_group, it)) return;
  }
  const int head = it.head;
  // the tiles start at the first 1024-byte boundary after the small buffers; the check
  // tests that they fit whatever the base's alignment
  extern __shared__ uint8_t smem_raw[];
  float* sLse = reinterpret_cast<float*>(smem_raw);  // [QS][128]
  float* sDel = sLse + Geo::QS * 128;                // [OS][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sDel + Geo::OS * 128);
  uint64_t* kv_full = bars;                // [1]
  uint64_t* q_full = kv_full + 1;          // [QS] Q tile (TMA) and its lse (statistics warp)
  uint64_t* q_empty = q_full + Geo::QS;    // [QS]
  uint64_t* o_full = q_empty + Geo::QS;    // [OS] dO tile and its Delta
  uint64_t* o_empty = o_full + Geo::OS;    // [OS]
  uint64_t* s_full = o_empty + Geo::OS;    // scores of the current tile written
  uint64_t* g_full = s_full + 1;           // dP^T of the current tile written
  uint64_t* p_ready = g_full + 1;          // packed P^T stored (8 warps)
  uint64_t* g_taken = p_ready + 1;         // dP^T loaded into registers (8 warps)
  uint64_t* ds_ready = g_taken + 1;        // packed dS^T stored (8 warps)
  uint64_t* acc_done = ds_ready + 1;
  uint64_t* tail_q = acc_done + 1;         // the last Q tile is cleared behind the sequence
  uint64_t* tail_o = tail_q + 1;           // and the last dO tile
  uint64_t* drain = tail_o + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t base = smem_addr(smem_raw);
  const uint32_t tiles_off = ((base + Geo::SMALL + 1023u) & ~1023u) - base;
  if (tiles_off > Geo::TILES_OFF) {  // uniform
    if (threadIdx.x == 0) record_error(p.status, kStatusUnsupported, SITE_SMEM_LAYOUT);
    return;
  }
  uint8_t* sK = smem_raw + tiles_off;
  uint8_t* sV = sK + Geo::TILE_B;
  uint8_t* sQ0 = sV + Geo::TILE_B;               // [QS]
  uint8_t* sO0 = sQ0 + Geo::QS * Geo::TILE_B;    // [OS]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = it.q0;              // first key
  const int first = k0 / p.TPT;      // the first query tile that sees a key
  const int n_inner = (it.len - 1) / p.TPT + 1 - first;
  const bool ragged = (first + n_inner) * p.TPT > it.len;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < Geo::QS; ++s) {
      mbar_init(&q_full[s], 2);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < Geo::OS; ++s) {
      mbar_init(&o_full[s], 2);
      mbar_init(&o_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(g_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(g_taken, 8);
    mbar_init(ds_ready, 8);
    mbar_init(acc_done, 1);
    mbar_init(tail_q, 1);
    mbar_init(tail_o, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // K and V are under way while the CTA sets itself up
    mbar_arrive_expect_tx(kv_full, 2 * Geo::TILE_B);
#pragma unroll
    for (int b = 0; b < Geo::BOXES; ++b) {
      tma_load_2d(sK + b * BOX_BYTES, &tmK, kv_full, head * HD + 64 * b, it.start + k0);
      tma_load_2d(sV + b * BOX_BYTES, &tmV, kv_full, head * HD + 64 * b, it.start + k0);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if (p.RU < 128) {
    // rows that no TMA box writes: zeros for the whole run
    for (int s = 0; s < Geo::QS + Geo::OS; ++s)
      clear_rows(sQ0 + s * Geo::TILE_B, Geo::BOXES, p.RU, threadIdx.x, Geo::THREADS);
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  WaitBound wb{p.status, p.limit_ns, abort_flag};
  const uint32_t box_rows = (uint32_t)(Geo::BOXES * 128) * (uint32_t)p.RU;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      int q_last[Geo::QS], o_last[Geo::OS];
      for (int s = 0; s < Geo::QS; ++s) q_last[s] = -1;
      for (int s = 0; s < Geo::OS; ++s) o_last[s] = -1;
      bool ok = true;
      for (int idx = 0; idx < n_inner; ++idx) {
        const int r0 = it.start + (first + idx) * p.TPT;
        const int qs = idx % Geo::QS, os = idx % Geo::OS;
        const uint32_t qph = (uint32_t)((idx / Geo::QS) & 1), oph = (uint32_t)((idx / Geo::OS) & 1);
        ok = mbar_wait(&q_empty[qs], qph ^ 1u, wb, SITE_PACKED_PRODUCER);
        if (!ok) break;
        mbar_arrive_expect_tx(&q_full[qs], box_rows);
#pragma unroll
        for (int b = 0; b < Geo::BOXES; ++b)
          tma_load_3d(sQ0 + qs * Geo::TILE_B + b * BOX_BYTES, &tmQ, &q_full[qs], 64 * b, head * p.G, r0);
        q_last[qs] = (int)qph;
        ok = mbar_wait(&o_empty[os], oph ^ 1u, wb, SITE_PACKED_PRODUCER);
        if (!ok) break;
        mbar_arrive_expect_tx(&o_full[os], box_rows);
#pragma unroll
        for (int b = 0; b < Geo::BOXES; ++b)
          tma_load_3d(sO0 + os * Geo::TILE_B + b * BOX_BYTES, &tmDO, &o_full[os], 64 * b, head * p.G, r0);
        o_last[os] = (int)oph;
      }
      // copies in flight land before the CTA ends. After a wait that gave up, the
      // statistics warp may have left a phase without its arrival: these waits then end
      // at their bound.
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(kv_full, 0, wd, SITE_DRAIN);
      for (int s = 0; s < Geo::QS; ++s)
        if (q_last[s] >= 0) mbar_wait(&q_full[s], (uint32_t)q_last[s], wd, SITE_DRAIN);
      for (int s = 0; s < Geo::OS; ++s)
        if (o_last[s] >= 0) mbar_wait(&o_full[s], (uint32_t)o_last[s], wd, SITE_DRAIN);
    }
  } else if (warp == 10) {
    // -------------------------------------------------------------- statistics
    // lse and Delta of each streamed tile: row r = token * G + head; four rows per lane,
    // fetched a tile ahead
    const float* lse_h = p.lse + (long long)head * p.G * p.ld_lse + it.start;
    const float* del_h = p.delta + (long long)head * p.G * p.ld_delta + it.start;
    float ls[4], de[4];
    auto fetch = [&](int idx) {
      const int t0 = (first + idx) * p.TPT;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = u * 32 + lane, tok = r / p.G, g = r - tok * p.G;
        const bool is = r < p.RU && t0 + tok < it.len;
        ls[u] = is ? lse_h[(long long)g * p.ld_lse + t0 + tok] : INFINITY;
        de[u] = is ? del_h[(long long)g * p.ld_delta + t0 + tok] : 0.f;
      }
    };
    fetch(0);
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, wb, SITE_PACKED_PRODUCER)) != 0;
    };
    for (int idx = 0; ok && idx < n_inner; ++idx) {
      const int qs = idx % Geo::QS, os = idx % Geo::OS;
      const uint32_t qph = (uint32_t)((idx / Geo::QS) & 1), oph = (uint32_t)((idx / Geo::OS) & 1);
      ok = warp_wait(&q_empty[qs], qph ^ 1u);
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < 4; ++u) sLse[qs * 128 + u * 32 + lane] = ls[u];
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qs]);
      ok = warp_wait(&o_empty[os], oph ^ 1u);
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < 4; ++u) sDel[os * 128 + u * 32 + lane] = de[u];
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_full[os]);
      if (idx + 1 < n_inner) fetch(idx + 1);
    }
    if (ok && ragged) {
      const int last = n_inner - 1;
      const int keep = (it.len - (first + last) * p.TPT) * p.G;  // rows of the sequence
      const int qs = last % Geo::QS, os = last % Geo::OS;
      if (warp_wait(&q_full[qs], (uint32_t)((last / Geo::QS) & 1))) {
        clear_rows(sQ0 + qs * Geo::TILE_B, Geo::BOXES, keep, lane, 32);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(tail_q);
        if (warp_wait(&o_full[os], (uint32_t)((last / Geo::OS) & 1))) {
          clear_rows(sO0 + os * Geo::TILE_B, Geo::BOXES, keep, lane, 32);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(tail_o);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc_s = make_idesc_bf16(TILE, TILE, false);
      const uint32_t idesc_acc = make_idesc_bf16(TILE, HD, true);
      const uint64_t dk0 = make_sdesc_sw128(smem_addr(sK), 16, 1024);
      const uint64_t dv0 = make_sdesc_sw128(smem_addr(sV), 16, 1024);
      const uint64_t dq0 = make_sdesc_sw128(smem_addr(sQ0), 16, 1024);            // K-major
      const uint64_t dq0_mn = make_sdesc_sw128(smem_addr(sQ0), BOX_BYTES, 1024);  // MN-major
      const uint64_t do0 = make_sdesc_sw128(smem_addr(sO0), 16, 1024);
      const uint64_t do0_mn = make_sdesc_sw128(smem_addr(sO0), BOX_BYTES, 1024);
      const uint32_t k_lo = (uint32_t)dk0, k_hi = (uint32_t)(dk0 >> 32);
      const uint32_t v_lo = (uint32_t)dv0, v_hi = (uint32_t)(dv0 >> 32);
      const uint32_t kq_hi = (uint32_t)(dq0 >> 32), mn_hi = (uint32_t)(dq0_mn >> 32);
      auto issue_s = [&](int j) {
        const uint32_t q_lo = (uint32_t)dq0 + (uint32_t)(j % Geo::QS) * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss_w(tmem + tm_s(j), k_lo + kmajor_step(kk), k_hi, q_lo + kmajor_step(kk), kq_hi,
                   idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(s_full);
      };
      auto issue_g = [&](int j) {
        const uint32_t o_lo = (uint32_t)do0 + (uint32_t)(j % Geo::OS) * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss_w(tmem + tm_g(j), v_lo + kmajor_step(kk), v_hi, o_lo + kmajor_step(kk), kq_hi,
                   idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(g_full);
      };
      auto issue_dv = [&](int j) {
        const uint32_t o_lo = (uint32_t)do0_mn + (uint32_t)(j % Geo::OS) * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          mma_ts_w(tmem + 0, tmem + packed_step(tm_s(j), kk), o_lo + (uint32_t)(kk * 128), mn_hi,
                   idesc_acc, (j == 0 && kk == 0) ? 0u : 1u);
      };
      auto issue_dk = [&](int j) {
        const uint32_t q_lo = (uint32_t)dq0_mn + (uint32_t)(j % Geo::QS) * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          mma_ts_w(tmem + HD, tmem + packed_step(tm_s(j) + 32, kk), q_lo + (uint32_t)(kk * 128),
                   mn_hi, idesc_acc, (j == 0 && kk == 0) ? 0u : 1u);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_poll(bar, parity, wb, SITE_PACKED_MMA);
      };
      // tile j's Q (dO) is in shared memory, and cleared where it is the ragged last one
      auto wait_q = [&](int j) {
        return wait(&q_full[j % Geo::QS], (uint32_t)((j / Geo::QS) & 1)) &&
               (!ragged || j != n_inner - 1 || wait(tail_q, 0));
      };
      auto wait_o = [&](int j) {
        return wait(&o_full[j % Geo::OS], (uint32_t)((j / Geo::OS) & 1)) &&
               (!ragged || j != n_inner - 1 || wait(tail_o, 0));
      };
      bool ok = wait(kv_full, 0) && wait_q(0);
      if (ok) {
        tc_fence_after();
        issue_s(0);
      }
      ok = ok && wait_o(0);
      if (ok) {
        tc_fence_after();
        issue_g(0);
      }
      // per tile j: dV(j) once P^T(j) is stored; S^T(j+1) into the dP^T(j) region once the
      // element-wise warps hold dP^T(j); dK(j) once dS^T(j) is stored; dP^T(j+1) into the
      // region of tile j, after dV(j) and dK(j) have read it (in issue order)
      for (int j = 0; ok && j < n_inner; ++j) {
        const uint32_t ph = (uint32_t)(j & 1);
        const bool more = j + 1 < n_inner;
        ok = wait(p_ready, ph);
        if (!ok) break;
        tc_fence_after();
        issue_dv(j);
        if (more) {
          ok = wait(g_taken, ph) && wait_q(j + 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(j + 1);
        }
        ok = wait(ds_ready, ph);
        if (!ok) break;
        tc_fence_after();
        issue_dk(j);
        mma_commit(&q_empty[j % Geo::QS]);
        mma_commit(&o_empty[j % Geo::OS]);
        if (more) {
          ok = wait_o(j + 1);
          if (!ok) break;
          tc_fence_after();
          issue_g(j + 1);
        }
      }
      if (ok) mma_commit(acc_done);
      mma_commit(drain);
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(drain, 0, wd, SITE_DRAIN);
    }
  } else {
    // -------------------------------------------------------------- element-wise
    const int g = (warp - 2) >> 2;  // query rows [64g, 64g + 64) of every tile
    const int qq = warp & 3;        // TMEM lane quarter
    const int kp = k0 + qq * 32 + lane;  // this thread's key, as a position of the sequence
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      const bool mine = mbar_wait(bar, parity, wb, SITE_PACKED_SOFTMAX);
      return __all_sync(0xffffffffu, mine) != 0;
    };
    for (int j = 0; j < n_inner; ++j) {
      const uint32_t ph = (uint32_t)(j & 1);
      const int qs = j % Geo::QS, os = j % Geo::OS;
      if (!warp_wait(s_full, ph) || !warp_wait(&q_full[qs], (uint32_t)((j / Geo::QS) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_t = lane_base + tm_s(j) + (uint32_t)(GCOLS * g);
      const uint32_t g_t = lane_base + tm_g(j) + (uint32_t)(GCOLS * g);
      uint32_t sv[2][32];
      tmem_ld32(s_t, sv[0]);
      tmem_ld32(s_t + 32, sv[1]);
      const float4* sl4 = reinterpret_cast<const float4*>(sLse + qs * 128 + g * GCOLS);
      // row c of the tile is the query at token t0 + c / G: it sees this key iff
      // c >= (kp - t0) G
      const int t0 = (first + j) * p.TPT;
      const bool masked = t0 < k0 + TILE - 1;
      const int c_min = max(kp - t0, 0) * p.G - g * GCOLS;
      tmem_ld_wait();
      // P^T = exp2(s * scale_log2 - lse[q]), kept in fp32 for dS^T and stored as bf16
      float pf[64];
      uint32_t pp[32];
      auto p_chunk = [&](const uint32_t (&s)[32], int c0, auto mask_tag) {
        constexpr bool MASK = decltype(mask_tag)::value;
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l4 = sl4[(c0 + e) >> 2];
          const uint64_t nl[2] = {f2_pack(-l4.x, -l4.y), f2_pack(-l4.z, -l4.w)};
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e + u]), __uint_as_float(s[e + u + 1])),
                             scale2, nl[u >> 1]),
                      x0, x1);
            float p0 = ex2(x0), p1 = ex2(x1);
            if constexpr (MASK) {
              p0 = c0 + e + u >= c_min ? p0 : 0.f;
              p1 = c0 + e + u + 1 >= c_min ? p1 : 0.f;
            }
            pf[c0 + e + u] = p0;
            pf[c0 + e + u + 1] = p1;
            pp[(c0 + e + u) >> 1] = pack_bf16x2(p0, p1);
          }
        }
      };
      if (masked) {
        p_chunk(sv[0], 0, std::true_type{});
        p_chunk(sv[1], 32, std::true_type{});
      } else {
        p_chunk(sv[0], 0, std::false_type{});
        p_chunk(sv[1], 32, std::false_type{});
      }
      tmem_st32(s_t, pp);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);
      if (!warp_wait(g_full, ph) || !warp_wait(&o_full[os], (uint32_t)((j / Geo::OS) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t gv[2][32];
      tmem_ld32(g_t, gv[0]);
      tmem_ld32(g_t + 32, gv[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(g_taken);
      // dS^T = P^T (dP^T - Delta[q])
      const float4* sd4 = reinterpret_cast<const float4*>(sDel + os * 128 + g * GCOLS);
      auto ds_chunk = [&](int c, auto mask_tag) {
        constexpr bool MASK = decltype(mask_tag)::value;
        uint32_t dd[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d4 = sd4[(32 * c + e) >> 2];
          const uint64_t dl[2] = {f2_pack(d4.x, d4.y), f2_pack(d4.z, d4.w)};
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            float d0, d1;
            f2_unpack(f2_mul(f2_pack(pf[32 * c + e + u], pf[32 * c + e + u + 1]),
                             f2_sub(f2_pack(__uint_as_float(gv[c][e + u]),
                                            __uint_as_float(gv[c][e + u + 1])),
                                    dl[u >> 1])),
                      d0, d1);
            if constexpr (MASK) {  // 0 times a dP that is not finite is not 0
              d0 = 32 * c + e + u >= c_min ? d0 : 0.f;
              d1 = 32 * c + e + u + 1 >= c_min ? d1 : 0.f;
            }
            dd[(e + u) >> 1] = pack_bf16x2(d0, d1);
          }
        }
        tmem_st16(s_t + 32 + 16 * c, dd);
      };
      if (masked) {
        ds_chunk(0, std::true_type{});
        ds_chunk(1, std::true_type{});
      } else {
        ds_chunk(0, std::false_type{});
        ds_chunk(1, std::false_type{});
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && warp_wait(acc_done, 0u)) {
      tc_fence_after();
      const bool row_ok = kp < it.len;
      const long long row = (long long)it.start + (row_ok ? kp : 0);
      __nv_bfloat16* dvp = p.dv + row * p.ld_dv + head * HD;
      __nv_bfloat16* dkp = p.dk + row * p.ld_dk + head * HD;
#pragma unroll
      for (int c = g * (HD / 2); c < (g + 1) * (HD / 2); c += 32) {
        uint32_t a[32], b[32];
        tmem_ld32(lane_base + (uint32_t)c, a);
        tmem_ld32(lane_base + (uint32_t)(HD + c), b);
        tmem_ld_wait();
        if (row_ok) {
          uint4* v4 = reinterpret_cast<uint4*>(dvp + c);
          uint4* k4 = reinterpret_cast<uint4*>(dkp + c);
          auto pair = [](const uint32_t* r, float f) {
            return pack_bf16x2(__uint_as_float(r[0]) * f, __uint_as_float(r[1]) * f);
          };
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            v4[w] = make_uint4(pair(a + 8 * w, 1.f), pair(a + 8 * w + 2, 1.f), pair(a + 8 * w + 4, 1.f),
                               pair(a + 8 * w + 6, 1.f));
            k4[w] = make_uint4(pair(b + 8 * w, p.scale), pair(b + 8 * w + 2, p.scale),
                               pair(b + 8 * w + 4, p.scale), pair(b + 8 * w + 6, p.scale));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ============================================================== query side
template <int HD>
__global__ void __launch_bounds__(QueryGeom<HD>::THREADS, 1)
    packed_bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmDO,
                         const __grid_constant__ CUtensorMap tmO,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const BwdParams p) {
  using Geo = QueryGeom<HD>;
  constexpr int NS = Geo::KV_STAGES;
  Item it;
  {
    const int per_group = p.src.max_items * p.src.group;
    const int grp = (int)blockIdx.x / per_group;
    if (!find_item(p.src, grp, (int)blockIdx.x - grp * per_group, it)) return;
  }
  const int head = it.head;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sStage = smem;  // stage s: K, V
  // the owned rows on their way to TMEM, in the stages that the ring does not use yet
  uint8_t* sQ = sStage + Geo::STAGE;
  uint8_t* sDO = sQ + Geo::TILE_B;
  uint8_t* sO = sStage + 2 * Geo::STAGE;
  float* sDel = reinterpret_cast<float*>(sStage + NS * Geo::STAGE);  // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sDel + 256);
  uint64_t* own_full = bars;         // Q, dO and o tiles in shared memory
  uint64_t* a_full = own_full + 1;   // Q and dO rows stored in TMEM (8 warps)
  uint64_t* kv_full = a_full + 1;    // [NS]
  uint64_t* kv_empty = kv_full + NS; // [NS]
  uint64_t* s_full = kv_empty + NS;  // S(j) in TMEM
  uint64_t* dp_full = s_full + 1;    // dP(j) in TMEM
  uint64_t* s_free = dp_full + 1;    // S(j) read by the element-wise warps (8)
  uint64_t* ds_full = s_free + 1;    // dS(j) stored (8 warps)
  uint64_t* acc_done = ds_full + 1;
  uint64_t* del_full = acc_done + 1; // both halves of a direct Delta stored (8)
  uint64_t* tail_ok = del_full + 1;  // the last K, V tiles are cleared behind the sequence
  uint64_t* drain = tail_ok + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_tiles = (min(it.len, it.q0 + p.TPT) - 1) / TILE + 1;
  const bool ragged = n_tiles * TILE > it.len;
  // Delta from o, or, where one tile holds all keys, from P and dP themselves: there o is a
  // mean of few values, and its rounding would be the largest error of dS
  const bool direct = n_tiles == 1;

  if (threadIdx.x == 0) {
    mbar_init(own_full, 1);
    mbar_init(a_full, 8);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(s_free, 8);
    mbar_init(ds_full, 8);
    mbar_init(acc_done, 1);
    mbar_init(del_full, 8);
    mbar_init(tail_ok, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // the owned rows and the first keys are under way while the CTA sets itself up
    mbar_arrive_expect_tx(own_full, (uint32_t)(Geo::BOXES * 128) * (uint32_t)p.RU * (direct ? 2u : 3u));
    mbar_arrive_expect_tx(&kv_full[0], 2 * Geo::TILE_B);
#pragma unroll
    for (int b = 0; b < Geo::BOXES; ++b) {
      tma_load_3d(sQ + b * BOX_BYTES, &tmQ, own_full, 64 * b, head * p.G, it.start + it.q0);
      tma_load_3d(sDO + b * BOX_BYTES, &tmDO, own_full, 64 * b, head * p.G, it.start + it.q0);
      if (!direct) tma_load_3d(sO + b * BOX_BYTES, &tmO, own_full, 64 * b, head * p.G, it.start + it.q0);
      tma_load_2d(sStage + b * BOX_BYTES, &tmK, &kv_full[0], head * HD + 64 * b, it.start);
      tma_load_2d(sStage + Geo::TILE_B + b * BOX_BYTES, &tmV, &kv_full[0], head * HD + 64 * b, it.start);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  WaitBound wb{p.status, p.limit_ns, abort_flag};

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    bool all = true;
    if (lane == 0) {
      int last[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) last[s] = -1;
      last[0] = 0;
      // the other stages hold the owned rows until these are in TMEM
      if (n_tiles > 1) all = mbar_wait(a_full, 0, wb, SITE_PACKED_PRODUCER);
      for (int j = 1; all && j < n_tiles; ++j) {
        const int st = j % NS;
        const uint32_t ph = (uint32_t)((j / NS) & 1);
        if (!mbar_wait(&kv_empty[st], ph ^ 1u, wb, SITE_PACKED_PRODUCER)) {
          all = false;
          break;
        }
        mbar_arrive_expect_tx(&kv_full[st], 2 * Geo::TILE_B);
        uint8_t* sk = sStage + st * Geo::STAGE;
#pragma unroll
        for (int b = 0; b < Geo::BOXES; ++b) {
          tma_load_2d(sk + b * BOX_BYTES, &tmK, &kv_full[st], head * HD + 64 * b, it.start + j * TILE);
          tma_load_2d(sk + Geo::TILE_B + b * BOX_BYTES, &tmV, &kv_full[st], head * HD + 64 * b,
                      it.start + j * TILE);
        }
        last[st] = (int)ph;
      }
      WaitBound wd{p.status, p.limit_ns, nullptr};
      all = mbar_wait(own_full, 0, wd, SITE_DRAIN) && all;
      for (int s = 0; s < NS; ++s)
        if (last[s] >= 0) all = mbar_wait(&kv_full[s], (uint32_t)last[s], wd, SITE_DRAIN) && all;
    }
    all = __shfl_sync(0xffffffffu, all ? 1 : 0, 0) != 0;
    if (ragged && all) {
      const int st = (n_tiles - 1) % NS;
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(&kv_full[st], (uint32_t)(((n_tiles - 1) / NS) & 1), wd, SITE_DRAIN);
      const int keep = it.len - (n_tiles - 1) * TILE;
      clear_rows(sStage + st * Geo::STAGE, 2 * Geo::BOXES, keep, lane, 32);  // K, then V
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(tail_ok);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc_s = make_idesc_bf16(TILE, TILE, false);
      const uint32_t idesc_acc = make_idesc_bf16(TILE, HD, true);
      const uint64_t dst0 = make_sdesc_sw128(smem_addr(sStage), 16, 1024);
      const uint64_t dst0_mn = make_sdesc_sw128(smem_addr(sStage), BOX_BYTES, 1024);
      const uint32_t st_lo = (uint32_t)dst0, st_hi = (uint32_t)(dst0 >> 32);
      const uint32_t mn_lo = (uint32_t)dst0_mn, mn_hi = (uint32_t)(dst0_mn >> 32);
      auto issue_s = [&](int st) {
        const uint32_t k_lo = st_lo + (uint32_t)st * Geo::STAGE / 16;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ts_w(tmem + TM_SC, tmem + Geo::TM_Q + (uint32_t)(kk * 8), k_lo + kmajor_step(kk),
                   st_hi, idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(s_full);
      };
      auto issue_dp = [&](int st) {
        const uint32_t v_lo = st_lo + ((uint32_t)st * Geo::STAGE + Geo::TILE_B) / 16;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ts_w(tmem + TM_DP, tmem + Geo::TM_DO + (uint32_t)(kk * 8), v_lo + kmajor_step(kk),
                   st_hi, idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(dp_full);
      };
      auto issue_dq = [&](int st, bool first) {
        const uint32_t k_lo = mn_lo + (uint32_t)st * Geo::STAGE / 16;
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          mma_ts_w(tmem + 0, packed_step(tmem + TM_DP, kk), k_lo + (uint32_t)(kk * 128), mn_hi,
                   idesc_acc, (first && kk == 0) ? 0u : 1u);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_poll(bar, parity, wb, SITE_PACKED_MMA);
      };
      auto wait_kv = [&](int j) {
        return wait(&kv_full[j % NS], (uint32_t)((j / NS) & 1)) &&
               (!ragged || j != n_tiles - 1 || wait(tail_ok, 0));
      };
      bool ok = wait(a_full, 0) && wait_kv(0);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        issue_dp(0);
      }
      for (int j = 0; ok && j < n_tiles; ++j) {
        const int st = j % NS;
        const uint32_t ph = (uint32_t)(j & 1);
        if (j + 1 < n_tiles) {
          // next scores as soon as the element-wise warps hold this tile's
          ok = wait_kv(j + 1) && wait(s_free, ph);
          if (!ok) break;
          tc_fence_after();
          issue_s((j + 1) % NS);
        }
        ok = wait(ds_full, ph);
        if (!ok) break;
        tc_fence_after();
        issue_dq(st, j == 0);
        mma_commit(&kv_empty[st]);
        if (j + 1 < n_tiles) issue_dp((j + 1) % NS);
      }
      if (ok) mma_commit(acc_done);
      mma_commit(drain);
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(drain, 0, wd, SITE_DRAIN);
    }
  } else {
    // -------------------------------------------------------------- element-wise
    const int g = (warp - 2) >> 2;  // key half of every streamed tile this warpgroup takes
    const int qq = warp & 3;
    const int r_local = qq * 32 + lane;
    const int tok = r_local / p.G;
    const bool row_ok = r_local < p.RU && it.q0 + tok < it.len;
    const int qpos = row_ok ? it.q0 + tok : -1;
    const long long row = (long long)it.start + (row_ok ? qpos : 0);
    const int qh = row_ok ? head * p.G + (r_local - tok * p.G) : 0;
    const float lse = row_ok ? p.lse[(long long)qh * p.ld_lse + row] : INFINITY;
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint32_t s_t = lane_base + TM_SC + (uint32_t)(g * GCOLS);
    const uint32_t d_t = lane_base + TM_DP + (uint32_t)(g * GCOLS);
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      const bool mine = mbar_wait(bar, parity, wb, SITE_PACKED_SOFTMAX);
      return __all_sync(0xffffffffu, mine) != 0;
    };
    float del = 0.f;
    ok = warp_wait(own_full, 0u);
    if (ok) {
      // this thread's row of Q (warpgroup 0) or dO (warpgroup 1) into TMEM, two bf16 values
      // per column; warpgroup 1 also takes its row of o and forms Delta. Chunk c of row r
      // lies at chunk c ^ (r % 8) of its 128 bytes (the 128-byte swizzle).
      const uint32_t dst = lane_base + (g == 0 ? Geo::TM_Q : Geo::TM_DO);
      const uint4* src = reinterpret_cast<const uint4*>((g == 0 ? sQ : sDO) + r_local * 128);
      const uint4* os = reinterpret_cast<const uint4*>(sO + r_local * 128);
#pragma unroll
      for (int b = 0; b < Geo::BOXES; ++b) {
        uint32_t r[32];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const uint4 v = row_ok ? src[b * (BOX_BYTES / 16) + (w ^ (r_local & 7))] : make_uint4(0u, 0u, 0u, 0u);
          r[4 * w + 0] = v.x;
          r[4 * w + 1] = v.y;
          r[4 * w + 2] = v.z;
          r[4 * w + 3] = v.w;
        }
        tmem_st32(dst + (uint32_t)(32 * b), r);
        if (g == 1 && row_ok && !direct) {
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const uint4 v = os[b * (BOX_BYTES / 16) + (w ^ (r_local & 7))];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              del = fmaf(bf16_lo(u[e]), bf16_lo(r[4 * w + e]), del);
              del = fmaf(bf16_hi(u[e]), bf16_hi(r[4 * w + e]), del);
            }
          }
        }
      }
      if (g == 1) {
        sDel[r_local] = del;
        if (row_ok && !direct) p.delta[(long long)qh * p.ld_delta + row] = del;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full);
    }
    // all eight warps have stored their rows, and Delta with them
    ok = ok && warp_wait(a_full, 0u);
    del = sDel[r_local];
    for (int j = 0; ok && j < n_tiles; ++j) {
      const uint32_t ph = (uint32_t)(j & 1);
      if (!warp_wait(s_full, ph)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // ---- P of this query row for the group's 64 key columns
      float pf[64];
      {
        uint32_t s0[32], s1[32];
        tmem_ld32(s_t, s0);
        tmem_ld32(s_t + 32, s1);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          pf[c] = ex2(fmaf(__uint_as_float(s0[c]), p.scale_log2, -lse));
          pf[32 + c] = ex2(fmaf(__uint_as_float(s1[c]), p.scale_log2, -lse));
        }
      }
      const int kbase = j * TILE + g * GCOLS;
      // some key of the group is in the future of some row of the CTA
      const bool masked = kbase + GCOLS - 1 > qpos;
      if (masked) {
#pragma unroll
        for (int c = 0; c < 64; ++c) pf[c] = kbase + c <= qpos ? pf[c] : 0.f;
      }
      // ---- dS = P (dP - Delta)
      if (!warp_wait(dp_full, ph)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (direct) {
        float part = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t gv[32];
          tmem_ld32(d_t + (uint32_t)(32 * half), gv);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int c = 32 * half + e;
            if (kbase + c <= qpos) part = fmaf(pf[c], __uint_as_float(gv[e]), part);
          }
        }
        sDel[g * 128 + r_local] = part;
        __syncwarp();
        if (lane == 0) mbar_arrive(del_full);
        if (!warp_wait(del_full, 0u)) {
          ok = false;
          break;
        }
        del = sDel[r_local] + sDel[128 + r_local];
        if (g == 1 && row_ok) p.delta[(long long)qh * p.ld_delta + row] = del;
      }
      const uint64_t del2 = f2_pack(del, del);
      uint32_t dd[32];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t gv[32];
        tmem_ld32(d_t + (uint32_t)(32 * half), gv);
        tmem_ld_wait();
        if (masked) {  // 0 times a dP that is not finite is not 0
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (kbase + 32 * half + e > qpos) gv[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int c = 32 * half + e;
          float d0, d1;
          f2_unpack(f2_mul(f2_pack(pf[c], pf[c + 1]),
                           f2_sub(f2_pack(__uint_as_float(gv[e]), __uint_as_float(gv[e + 1])), del2)),
                    d0, d1);
          dd[c >> 1] = pack_bf16x2(d0, d1);
        }
      }
      tmem_st32(d_t, dd);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && warp_wait(acc_done, 0u)) {
      tc_fence_after();
      __nv_bfloat16* dqp = p.dq + row * p.ld_dq + (long long)qh * HD;
#pragma unroll
      for (int c = g * (HD / 2); c < (g + 1) * (HD / 2); c += 32) {
        uint32_t a[32];
        tmem_ld32(lane_base + (uint32_t)c, a);
        tmem_ld_wait();
        if (row_ok) {
          uint4* q4 = reinterpret_cast<uint4*>(dqp + c);
          auto pair = [&](int e) {
            return pack_bf16x2(__uint_as_float(a[e]) * p.scale, __uint_as_float(a[e + 1]) * p.scale);
          };
#pragma unroll
          for (int w = 0; w < 4; ++w)
            q4[w] = make_uint4(pair(8 * w), pair(8 * w + 2), pair(8 * w + 4), pair(8 * w + 6));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int HD>
tsp_status launch_bwd(const Shape& s, const Source& queries, const Source& keys, BwdParams p,
                      const void* k, int64_t ld_k, const void* v, int64_t ld_v, cudaStream_t stream) {
  CUtensorMap tq, tdo, to, tk, tv;
  TSP_TRY(make_query_map(&tq, s, p.q, p.ld_q));
  TSP_TRY(make_query_map(&tdo, s, p.dout, p.ld_do));
  TSP_TRY(make_query_map(&to, s, p.o, p.ld_o));
  const uint64_t cols = (uint64_t)s.kv_heads * HD, rows = (uint64_t)s.tokens;
  TSP_TRY(make_tmap_2d_bf16(&tk, k, cols, rows, (uint64_t)ld_k * 2, 64, TILE));
  TSP_TRY(make_tmap_2d_bf16(&tv, v, cols, rows, (uint64_t)ld_v * 2, 64, TILE));
  {
    auto kernel = packed_bwd_dq_kernel<HD>;
    const size_t smem = QueryGeom<HD>::SMEM;
    TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                              "packed attention backward: cudaFuncSetAttribute"));
    p.src = queries;
    kernel<<<(unsigned)p.src.max_items * (unsigned)s.kv_heads, QueryGeom<HD>::THREADS, smem, stream>>>(
        tq, tdo, to, tk, tv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "packed attention backward (query side): launch");
  }
  {
    auto kernel = packed_bwd_dkv_kernel<HD>;
    const size_t smem = KeyGeom<HD>::SMEM;
    TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                              "packed attention backward: cudaFuncSetAttribute"));
    p.src = keys;
    kernel<<<(unsigned)p.src.max_items * (unsigned)s.kv_heads, KeyGeom<HD>::THREADS, smem, stream>>>(
        tq, tdo, tk, tv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "packed attention backward (key side): launch");
  }
  return TSP_OK;
}

}  // namespace
}  // namespace packed
}  // namespace tsp

using namespace tsp;
using namespace tsp::packed;

extern "C" tsp_status tsp_packed_attention_bwd(
    int64_t tokens, int n_seqs, const int32_t* starts, int heads, int kv_heads, int head_dim,
    float scale, const tsp_bf16* q, int64_t ld_q, const tsp_bf16* k, int64_t ld_k, const tsp_bf16* v,
    int64_t ld_v, const tsp_bf16* o, int64_t ld_o, const float* lse, int64_t ld_lse,
    const tsp_bf16* dout, int64_t ld_do, tsp_bf16* dq, int64_t ld_dq, tsp_bf16* dk, int64_t ld_dk,
    tsp_bf16* dv, int64_t ld_dv, void* ws, void* stream) {
  const char* what = "tsp_packed_attention_bwd";
  Shape s;
  TSP_TRY(make_shape(what, tokens, n_seqs, heads, kv_heads, head_dim, &s));
  if (!(scale > 0.f) || !std::isfinite(scale))
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": scale must be positive and finite");
  if (tokens == 0 || n_seqs == 0) return TSP_OK;
  if (!starts || (reinterpret_cast<uintptr_t>(starts) & 3u))
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": starts is null or misaligned");
  const int64_t qc = (int64_t)heads * head_dim, kc = (int64_t)kv_heads * head_dim;
  TSP_TRY(check_matrix(what, "q", q, ld_q, qc));
  TSP_TRY(check_matrix(what, "k", k, ld_k, kc));
  TSP_TRY(check_matrix(what, "v", v, ld_v, kc));
  TSP_TRY(check_matrix(what, "o", o, ld_o, qc));
  TSP_TRY(check_matrix(what, "dout", dout, ld_do, qc));
  TSP_TRY(check_matrix(what, "dq", dq, ld_dq, qc));
  TSP_TRY(check_matrix(what, "dk", dk, ld_dk, kc));
  TSP_TRY(check_matrix(what, "dv", dv, ld_dv, kc));
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) || ld_lse < tokens)
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": lse null, misaligned, or its row stride below the tokens");
  const void* ins[] = {q, k, v, o, dout};
  const void* outs[] = {dq, dk, dv};
  for (const void* x : outs)
    for (const void* y : ins)
      if (x == y) return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": a gradient aliases an input");
  if (dq == dk || dq == dv || dk == dv)
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": two gradients alias");
  TSP_TRY(check_ws(ws, what));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Workspace w = make_workspace(s);
  auto in = [](const tsp_bf16* x) { return reinterpret_cast<const __nv_bfloat16*>(x); };
  auto out = [](tsp_bf16* x) { return reinterpret_cast<__nv_bfloat16*>(x); };
  BwdParams p{};
  p.dq = out(dq);
  p.dk = out(dk);
  p.dv = out(dv);
  p.ld_dq = ld_dq;
  p.ld_dk = ld_dk;
  p.ld_dv = ld_dv;
  p.q = in(q);
  p.o = in(o);
  p.dout = in(dout);
  p.ld_q = ld_q;
  p.ld_o = ld_o;
  p.ld_do = ld_do;
  p.lse = lse;
  p.ld_lse = ld_lse;
  p.delta = at<float>(ws, w.delta);
  p.ld_delta = w.ld_stat;
  p.G = s.G;
  p.TPT = s.TPT;
  p.RU = s.RU;
  p.scale_log2 = 1.4426950408889634f * scale;
  p.scale = scale;
  p.status = status_of(ws);
  p.limit_ns = wait_limit_ns();
  int* counts = at<int>(ws, w.counts);
  // 48 MB of K and V in L2 at a time, as for the plan's backward
  const int group = head_group(s, 48ll << 20);
  const Source queries = make_source(s, starts, s.TPT, false, group, at<Item>(ws, w.items), counts,
                                     (int)w.max_query, p.status);
  const Source keys = make_source(s, starts, TILE, true, group, at<Item>(ws, w.key_items), counts + 1,
                                  (int)w.max_key, p.status);
  if (queries.items != nullptr) {
    const ListArgs a{s.TPT, 0, list_shift((tokens + TILE - 1) / TILE), at<Item>(ws, w.items), counts,
                     (int)w.max_query};
    const ListArgs b{TILE, s.TPT, list_shift((tokens + s.TPT - 1) / s.TPT), at<Item>(ws, w.key_items),
                     counts + 1, (int)w.max_key};
    TSP_TRY(launch_lists(s, starts, a, b, p.status, st));
  }
  if (head_dim == 64) return launch_bwd<64>(s, queries, keys, p, k, ld_k, v, ld_v, st);
  return launch_bwd<128>(s, queries, keys, p, k, ld_k, v, ld_v, st);
}
