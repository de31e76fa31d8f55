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
// P and dS are rounded to bf16 as operands of the tensor core, at most 2^-8 of a term; dS is
// formed from the unrounded P. Accumulators and statistics are fp32. Delta from o takes the
// rounded o, off by at most 2^-8 sum |dO_ic o_ic|; with more than a tile of keys o is a mean of
// many values and that is small beside dS's own rounding (dq, dk and dv of 8192 packed tokens are
// off by 2.4e-3 in the two-norm, against 64 bits; their last rounding alone makes 1.7e-3).
// Both kernels are persistent as the forward is. The key side may start on multiprocessors
// that the query side has left; only its Delta waits for the end of that. Sequences of a few
// tokens go to no tile (packed_short.cuh).
//
// Rows that are no query of the sequence (the rows of a tile behind the sequence's end, and
// those past TPT x G when G does not divide 128) enter the key side's sums with P = 0: their
// lse is +infinity and their Q and dO rows are zeros in shared memory, so nothing that lies
// behind the sequence can reach a sum. The query side clears its last K and V tile the same
// way. Pairs above the diagonal are set to 0 by selection in P, and on the query side, where
// dP may hold a later key's infinity, in dS as well. On the key side selection in dS would not
// keep an earlier query's infinity out: 0 times its rows of Q and dO enters dK and dV all the
// same. So it reaches the later keys that share a tile with it: those below k0 + 128 for a key
// tile from k0 on, whose first query tile begins at floor(k0 / TPT) TPT.
//
// Measured, heads of 128: 16381 tokens, 32/4 heads 2.3 ms and 3.4 ms (1430 and 1300 TFLOP/s of
// the products that run); 8192 tokens in 27 sequences, 32/8 heads 0.15 and 0.16 ms (the 128 x
// 128 tiles hold 1.18 times the visible pairs, and an item's fill and epilogue cost about two
// tiles' time; tensor pipe 34 and 46% active, 0.30 and 0.26 instructions a cycle and scheduler, the
// warps waiting for loads, and d = 128 keeps 96 bytes a thread in local memory on the query side);
// 128 sequences of 128 tokens 0.14 and 0.11 ms (0.05 and 0.06 of it HBM).
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
#include "packed_short.cuh"

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
  const __nv_bfloat16* o;
  long long ld_o;
  const __nv_bfloat16* q;  // read directly for the short sequences
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* dout;
  long long ld_q, ld_k, ld_v, ld_do;
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

constexpr int ITEMS = 4;  // items between the producer and the slowest reader

template <int HD>
struct KeyGeom {
  static constexpr int THREADS = 352;  // TMA, MMA, 2 x 4 element-wise warps, statistics
  static constexpr int READERS = 10;   // of an item: MMA lane, statistics, 8 warps
  static constexpr int BOXES = HD / 64;
  static constexpr uint32_t TILE_B = 128 * HD * 2;
  // Q tiles (with lse) and dO tiles (with Delta) in separate rings: a Q tile is read last
  // by dK, a full tile after its scores, so it gets the deeper ring
  static constexpr int QS = 3;
  static constexpr int OS = 2;
  static constexpr uint32_t SMALL = (QS + OS) * 512 + ITEMS * 16 + 384;
  static constexpr uint32_t TILES_OFF = (SMALL + 1023) / 1024 * 1024;
  static constexpr size_t USED = TILES_OFF + (size_t)(2 + QS + OS) * TILE_B;
  static constexpr size_t SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
};
static_assert(KeyGeom<128>::USED <= 227 * 1024, "key-side shared memory");

template <int HD>
struct QueryGeom {
  static constexpr int THREADS = 320;
  static constexpr int READERS = 9;  // of an item: MMA lane, 8 warps
  static constexpr int BOXES = HD / 64;
  static constexpr uint32_t TILE_B = 128 * HD * 2;
  // a stage holds the item's Q and dO on their way to TMEM, or K and V of one key tile
  static constexpr int NS = 3;
  static constexpr uint32_t STAGE = 2 * TILE_B;
  static constexpr uint32_t SMALL = 1024 + ITEMS * 16 + 384;  // Delta, items, barriers
  static constexpr uint32_t TILES_OFF = (SMALL + 1023) / 1024 * 1024;
  static constexpr size_t USED = TILES_OFF + (size_t)NS * STAGE;
  static constexpr size_t SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr uint32_t TM_Q = HD;
  static constexpr uint32_t TM_DO = HD + HD / 2;
};
static_assert(QueryGeom<128>::USED <= 227 * 1024, "query-side shared memory");

// Offset of the tiles behind `small` bytes of a shared-memory base of any alignment; 0 if the
// allocation, made for `most`, has no room for them.
__device__ __forceinline__ uint32_t tiles_offset(const uint8_t* base, uint32_t small, uint32_t most) {
  const uint32_t at = smem_addr(base);
  const uint32_t off = ((at + small + 1023u) & ~1023u) - at;
  return off > most ? 0u : off;
}

// A millisecond, for copies that a wait which gave up may have left in flight.
__device__ __forceinline__ void let_copies_land() {
  const unsigned long long t0 = global_ns();
  while (global_ns() - t0 < 1000000ull) {
  }
}

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
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ BwdParams p) {
  using Geo = KeyGeom<HD>;
  constexpr uint32_t QS = Geo::QS, OS = Geo::OS;
  extern __shared__ uint8_t smem_raw[];
  float* sLse = reinterpret_cast<float*>(smem_raw);  // [QS][128]
  float* sDel = sLse + QS * 128;                     // [OS][128]
  Item* items = reinterpret_cast<Item*>(sDel + OS * 128);           // [ITEMS]
  uint64_t* item_full = reinterpret_cast<uint64_t*>(items + ITEMS); // [ITEMS]
  uint64_t* item_empty = item_full + ITEMS;  // [ITEMS]
  uint64_t* kv_full = item_empty + ITEMS;    // the item's K and V
  uint64_t* kv_empty = kv_full + 1;          // its S^T and dP^T are all computed
  uint64_t* q_full = kv_empty + 1;           // [QS] Q tile (TMA) and its lse (statistics warp)
  uint64_t* q_empty = q_full + QS;           // [QS]
  uint64_t* q_tail = q_empty + QS;           // [QS] a ragged Q tile is cleared behind the sequence
  uint64_t* o_full = q_tail + QS;            // [OS] dO tile and its Delta
  uint64_t* o_empty = o_full + OS;           // [OS]
  uint64_t* o_tail = o_empty + OS;           // [OS]
  uint64_t* s_full = o_tail + OS;            // scores of the current tile written
  uint64_t* g_full = s_full + 1;             // dP^T of the current tile written
  uint64_t* p_ready = g_full + 1;            // packed P^T stored (8 warps)
  uint64_t* g_taken = p_ready + 1;           // dP^T loaded into registers (8 warps)
  uint64_t* ds_ready = g_taken + 1;          // packed dS^T stored (8 warps)
  uint64_t* acc_done = ds_ready + 1;         // the item's dK and dV complete
  uint64_t* drain = acc_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t tiles_off = tiles_offset(smem_raw, Geo::SMALL, Geo::TILES_OFF);
  if (tiles_off == 0) {  // uniform
    if (threadIdx.x == 0) record_error(p.status, kStatusUnsupported, SITE_SMEM_LAYOUT);
    return;
  }
  uint8_t* sK = smem_raw + tiles_off;
  uint8_t* sV = sK + Geo::TILE_B;
  uint8_t* sQ0 = sV + Geo::TILE_B;        // [QS]
  uint8_t* sO0 = sQ0 + QS * Geo::TILE_B;  // [OS]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ITEMS; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], Geo::READERS);
    }
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (uint32_t s = 0; s < QS; ++s) {
      mbar_init(&q_full[s], 2);
      mbar_init(&q_empty[s], 1);
      mbar_init(&q_tail[s], 1);
    }
    for (uint32_t s = 0; s < OS; ++s) {
      mbar_init(&o_full[s], 2);
      mbar_init(&o_empty[s], 1);
      mbar_init(&o_tail[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(g_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(g_taken, 8);
    mbar_init(ds_ready, 8);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmDO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  uint32_t tmem = 0;
  if (warp == 0) {
    __syncwarp();
    start_arrive<Geo::THREADS>();
  } else {
    if (warp == 1) {
      tmem_alloc(tmem_slot, TMEM_COLS);
      tmem_relinquish();
    }
    if (p.RU < 128) {
      // rows that no TMA box writes: zeros for the whole run
      for (uint32_t s = 0; s < QS + OS; ++s)
        clear_rows(sQ0 + s * Geo::TILE_B, Geo::BOXES, p.RU, threadIdx.x - 32, Geo::THREADS - 32);
      fence_proxy_async();
    }
    tc_fence_before();
    start_sync<Geo::THREADS>();
    tc_fence_after();
    tmem = *tmem_slot;
  }
  WaitBound wb{p.status, p.limit_ns, abort_flag};
  // streamed query tiles of an item: from the first that sees one of its keys
  auto first_of = [&](const Item& it) { return it.q0 / p.TPT; };
  auto inner_of = [&](const Item& it) { return (it.len - 1) / p.TPT + 1 - it.q0 / p.TPT; };

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    const uint32_t box_rows = (uint32_t)(Geo::BOXES * 128) * (uint32_t)p.RU;
    Item next{};
    Walk walk;
    walk.next(p.src, next);
    bool ok = true;
    uint32_t n_items = 0, c = 0;  // items and streamed tiles so far
    while (ok) {
      const Item it = next;
      const int slot = (int)(n_items % ITEMS);
      if (lane == 0) {
        ok = mbar_wait(&item_empty[slot], ((n_items / ITEMS) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
        if (ok) {
          items[slot] = it;
          mbar_arrive(&item_full[slot]);
        }
        if (ok && it.head >= 0) {
          ok = mbar_wait(kv_empty, (n_items & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
          if (ok) {
            mbar_arrive_expect_tx(kv_full, 2 * Geo::TILE_B);
#pragma unroll
            for (int b = 0; b < Geo::BOXES; ++b) {
              tma_load_2d(sK + b * BOX_BYTES, &tmK, kv_full, it.head * HD + 64 * b, it.start + it.q0);
              tma_load_2d(sV + b * BOX_BYTES, &tmV, kv_full, it.head * HD + 64 * b, it.start + it.q0);
            }
          }
          const int n = inner_of(it);
          int r0 = it.start + first_of(it) * p.TPT;
          for (int j = 0; ok && j < n; ++j, ++c, r0 += p.TPT) {
            const uint32_t qs = c % QS, os = c % OS;
            ok = mbar_wait(&q_empty[qs], ((c / QS) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
            if (!ok) break;
            mbar_arrive_expect_tx(&q_full[qs], box_rows);
#pragma unroll
            for (int b = 0; b < Geo::BOXES; ++b)
              tma_load_3d(sQ0 + qs * Geo::TILE_B + b * BOX_BYTES, &tmQ, &q_full[qs], 64 * b,
                          it.head * p.G, r0);
            ok = mbar_wait(&o_empty[os], ((c / OS) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
            if (!ok) break;
            mbar_arrive_expect_tx(&o_full[os], box_rows);
#pragma unroll
            for (int b = 0; b < Geo::BOXES; ++b)
              tma_load_3d(sO0 + os * Geo::TILE_B + b * BOX_BYTES, &tmDO, &o_full[os], 64 * b,
                          it.head * p.G, r0);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok || it.head < 0) break;
      ++n_items;
      walk.next(p.src, next);
    }
    if (lane == 0) {
      walk.end(p.src);
      prior_kernel_done();  // this kernel ends after the query side, items or none
      // copies in flight land before the CTA ends
      WaitBound wd{p.status, p.limit_ns, nullptr};
      if (n_items > 0) mbar_wait(kv_full, (n_items - 1) & 1u, wd, SITE_DRAIN);
      for (uint32_t b = c > QS ? c - QS : 0; b < c; ++b)
        mbar_wait(&q_full[b % QS], (b / QS) & 1u, wd, SITE_DRAIN);
      for (uint32_t b = c > OS ? c - OS : 0; b < c; ++b)
        mbar_wait(&o_full[b % OS], (b / OS) & 1u, wd, SITE_DRAIN);
      if (!ok) let_copies_land();
    }
  } else if (warp == 10) {
    // -------------------------------------------------------------- statistics
    // lse and Delta of each streamed tile, row r = token * G + head, four rows per lane,
    // fetched a tile ahead; then zeros behind the sequence in its last Q and dO tiles
    bool ok = true;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, wb, SITE_PACKED_PRODUCER)) != 0;
    };
    prior_kernel_done();  // the query side has left Delta
    uint32_t n_items = 0, c = 0;
    while (ok) {
      const int slot = (int)(n_items % ITEMS);
      if (!warp_wait(&item_full[slot], n_items / ITEMS)) break;
      ++n_items;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      if (it.head < 0) break;
      const int n = inner_of(it);
      const float* lse_h = p.lse + (long long)it.head * p.G * p.ld_lse + it.start;
      const float* del_h = p.delta + (long long)it.head * p.G * p.ld_delta + it.start;
      float ls[4], de[4];
      auto fetch = [&](int t0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = u * 32 + lane, tok = r / p.G, g = r - tok * p.G;
          const bool is = r < p.RU && t0 + tok < it.len;
          ls[u] = is ? lse_h[(long long)g * p.ld_lse + t0 + tok] : INFINITY;
          de[u] = is ? del_h[(long long)g * p.ld_delta + t0 + tok] : 0.f;
        }
      };
      int t0 = first_of(it) * p.TPT;
      fetch(t0);
      for (int j = 0; ok && j < n; ++j, ++c, t0 += p.TPT) {
        const uint32_t qs = c % QS, os = c % OS;
        ok = warp_wait(&q_empty[qs], (c / QS) ^ 1u);
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) sLse[qs * 128 + u * 32 + lane] = ls[u];
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[qs]);
        ok = warp_wait(&o_empty[os], (c / OS) ^ 1u);
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) sDel[os * 128 + u * 32 + lane] = de[u];
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_full[os]);
        if (j + 1 < n) fetch(t0 + p.TPT);
      }
      // rows of the sequence in the item's last tile
      const int keep = (it.len - (t0 - p.TPT)) * p.G;
      if (ok && keep < p.RU) {
        const uint32_t last = c - 1;
        const uint32_t qs = last % QS, os = last % OS;
        ok = warp_wait(&q_full[qs], last / QS);
        if (!ok) break;
        clear_rows(sQ0 + qs * Geo::TILE_B, Geo::BOXES, keep, lane, 32);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_tail[qs]);
        ok = warp_wait(&o_full[os], last / OS);
        if (!ok) break;
        clear_rows(sO0 + os * Geo::TILE_B, Geo::BOXES, keep, lane, 32);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_tail[os]);
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
      // c: streamed tiles so far, over all items; qs, os: their stages
      auto issue_s = [&](uint32_t c, uint32_t qs) {
        const uint32_t q_lo = (uint32_t)dq0 + qs * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss_w(tmem + tm_s((int)c), k_lo + kmajor_step(kk), k_hi, q_lo + kmajor_step(kk), kq_hi,
                   idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(s_full);
      };
      auto issue_g = [&](uint32_t c, uint32_t os) {
        const uint32_t o_lo = (uint32_t)do0 + os * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss_w(tmem + tm_g((int)c), v_lo + kmajor_step(kk), v_hi, o_lo + kmajor_step(kk), kq_hi,
                   idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(g_full);
      };
      auto issue_dv = [&](uint32_t c, uint32_t os, bool first) {
        const uint32_t o_lo = (uint32_t)do0_mn + os * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          mma_ts_w(tmem + 0, tmem + packed_step(tm_s((int)c), kk), o_lo + (uint32_t)(kk * 128), mn_hi,
                   idesc_acc, (first && kk == 0) ? 0u : 1u);
      };
      auto issue_dk = [&](uint32_t c, uint32_t qs, bool first) {
        const uint32_t q_lo = (uint32_t)dq0_mn + qs * (Geo::TILE_B / 16);
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          mma_ts_w(tmem + HD, tmem + packed_step(tm_s((int)c) + 32, kk), q_lo + (uint32_t)(kk * 128),
                   mn_hi, idesc_acc, (first && kk == 0) ? 0u : 1u);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_poll(bar, parity & 1u, wb, SITE_PACKED_MMA);
      };
      // The Q (dO) tile of a stage is in place, and cleared if it is its sequence's ragged last
      // one. Bit st of ph_q, ph_o, turn_q and turn_o is the phase of the stage's barrier.
      uint32_t ph_q = 0, ph_o = 0, turn_q = 0, turn_o = 0;
      auto landed = [&](uint64_t* full, uint64_t* tail, uint32_t st, uint32_t& ph, uint32_t& turn, bool ragged) {
        if (!wait(&full[st], ph >> st)) return false;
        ph ^= 1u << st;
        if (!ragged) return true;
        const bool ok = wait(&tail[st], turn >> st);
        turn ^= 1u << st;
        return ok;
      };
      auto wait_q = [&](uint32_t st, bool ragged) { return landed(q_full, q_tail, st, ph_q, turn_q, ragged); };
      auto wait_o = [&](uint32_t st, bool ragged) { return landed(o_full, o_tail, st, ph_o, turn_o, ragged); };
      bool ok = true;
      uint32_t n_items = 0, c = 0, qs = 0;
      while (ok) {
        const int slot = (int)(n_items % ITEMS);
        ok = wait(&item_full[slot], n_items / ITEMS);
        if (!ok) break;
        const Item it = items[slot];
        mbar_arrive(&item_empty[slot]);
        if (it.head < 0) break;
        const int n = inner_of(it);
        const bool ragged = (first_of(it) + n) * p.TPT > it.len;
        // S^T(c) goes over the dP^T(c - 1) of the item before, once that is in registers
        ok = wait(kv_full, n_items) && wait_q(qs, ragged && n == 1) && (c == 0 || wait(g_taken, c - 1));
        if (!ok) break;
        tc_fence_after();
        issue_s(c, qs);
        ok = wait_o(c % OS, ragged && n == 1);
        if (!ok) break;
        tc_fence_after();
        issue_g(c, c % OS);
        if (n == 1) mma_commit(kv_empty);
        // per tile: dV once P^T is stored; the next S^T into the dP^T region once the
        // element-wise warps hold dP^T; dK once dS^T is stored; the next dP^T into the
        // region of this tile, after dV and dK have read it (in issue order)
        for (int j = 0; j < n; ++j, ++c) {
          const bool more = j + 1 < n, last_next = ragged && j + 2 == n;
          const uint32_t os = c % OS, qn = qs + 1 == QS ? 0 : qs + 1;
          ok = wait(p_ready, c);
          if (!ok) break;
          tc_fence_after();
          issue_dv(c, os, j == 0);
          if (more) {
            ok = wait(g_taken, c) && wait_q(qn, last_next);
            if (!ok) break;
            tc_fence_after();
            issue_s(c + 1, qn);
          }
          ok = wait(ds_ready, c);
          if (!ok) break;
          tc_fence_after();
          issue_dk(c, qs, j == 0);
          mma_commit(&q_empty[qs]);
          mma_commit(&o_empty[os]);
          qs = qn;
          if (more) {
            ok = wait_o(os ^ 1u, last_next);
            if (!ok) break;
            tc_fence_after();
            issue_g(c + 1, os ^ 1u);
            if (j + 2 == n) mma_commit(kv_empty);
          }
        }
        if (ok) mma_commit(acc_done);
        ++n_items;
      }
      mma_commit(drain);
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(drain, 0, wd, SITE_DRAIN);
    }
  } else {
    // -------------------------------------------------------------- element-wise
    const int g = (warp - 2) >> 2;  // query rows [64g, 64g + 64) of every tile
    const int qq = warp & 3;        // TMEM lane quarter
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      const bool mine = mbar_wait(bar, parity & 1u, wb, SITE_PACKED_SOFTMAX);
      return __all_sync(0xffffffffu, mine) != 0;
    };
    // the short sequences, under the first item's loads
    short_key_side<HD>(p, (gridDim.x - 1u - blockIdx.x) * 8u + (unsigned)(warp - 2), gridDim.x * 8u);
    // The loop below is short of issue slots: stages, phases and addresses step along instead
    // of being computed from the tile's number (remainders by 3 alone cost 0.1 of 1.8 us a tile).
    uint32_t n_items = 0, c = 0;              // items and streamed tiles so far
    uint32_t qs = 0, qph = 0;                 // stage and phase of the Q ring
    uint32_t s_t = lane_base + tm_s(0) + (uint32_t)(GCOLS * g);  // this tile's scores
    uint32_t g_t = lane_base + tm_g(0) + (uint32_t)(GCOLS * g);  // and its dP^T
    while (true) {
      const int slot = (int)(n_items % ITEMS);
      if (!warp_wait(&item_full[slot], n_items / ITEMS)) break;
      // what the epilogue needs of the item is read again there, and only then is the slot
      // released: the loop below has no registers to spare
      int n, t0, kp;
      {
        const Item it = items[slot];
        if (it.head < 0) break;
        n = inner_of(it);
        t0 = first_of(it) * p.TPT;
        kp = it.q0 + qq * 32 + lane;  // this thread's key, as a position of the sequence
      }
      bool ok = true;
      for (int j = 0; j < n; ++j, ++c, t0 += p.TPT) {
        const uint32_t os = c & 1u;
        if (!warp_wait(s_full, c) || !warp_wait(&q_full[qs], qph)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sv[2][32];
        tmem_ld32(s_t, sv[0]);
        tmem_ld32(s_t + 32, sv[1]);
        const float4* sl4 = reinterpret_cast<const float4*>(sLse + qs * 128 + g * GCOLS);
        // row e of the tile is the query at token t0 + e / G: it sees this key iff
        // e >= (kp - t0) G
        const bool masked = t0 < kp - (qq * 32 + lane) + TILE - 1;
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
        if (!warp_wait(g_full, c) || !warp_wait(&o_full[os], c >> 1)) {
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
        // dS^T = P^T (dP^T - Delta[q]), 0 where P^T was set to 0
        const float4* sd4 = reinterpret_cast<const float4*>(sDel + os * 128 + g * GCOLS);
        auto ds_chunk = [&](int h) {
          uint32_t dd[16];
  #pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 d4 = sd4[(32 * h + e) >> 2];
            const uint64_t dl[2] = {f2_pack(d4.x, d4.y), f2_pack(d4.z, d4.w)};
  #pragma unroll
            for (int u = 0; u < 4; u += 2) {
              float d0, d1;
              f2_unpack(f2_mul(f2_pack(pf[32 * h + e + u], pf[32 * h + e + u + 1]),
                               f2_sub(f2_pack(__uint_as_float(gv[h][e + u]),
                                              __uint_as_float(gv[h][e + u + 1])),
                                      dl[u >> 1])),
                        d0, d1);
              dd[(e + u) >> 1] = pack_bf16x2(d0, d1);
            }
          }
          tmem_st16(s_t + 32 + 16 * h, dd);
        };
        ds_chunk(0);
        ds_chunk(1);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_ready);
        if (++qs == QS) {
          qs = 0;
          qph ^= 1u;
        }
        const uint32_t swap = s_t;
        s_t = g_t;
        g_t = swap;
      }
      if (!ok || !warp_wait(acc_done, n_items)) break;
      ++n_items;
      // ---------------------------------------------------------- epilogue
      // P^T of the next item is handed over after these loads, and only then may its first
      // products overwrite dV and dK
      tc_fence_after();
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      const bool row_ok = kp < it.len;
      const long long row = (long long)it.start + (row_ok ? kp : 0);
      auto store = [&](__nv_bfloat16* base, long long ld, uint32_t column, float f) {
        __nv_bfloat16* dst[4];
        group_rows(row_ok ? base + row * ld + it.head * HD + g * (HD / 2) : nullptr, dst);
#pragma unroll
        for (int e0 = 0; e0 < HD / 2; e0 += 32) {
          uint32_t r[32], w[16];
          tmem_ld32(lane_base + column + (uint32_t)(g * (HD / 2) + e0), r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * f, __uint_as_float(r[2 * e + 1]) * f);
          store_rows(w, dst);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (dst[k] != nullptr) dst[k] += 32;
        }
      };
      store(p.dv, p.ld_dv, 0u, 1.f);
      store(p.dk, p.ld_dk, (uint32_t)HD, p.scale);
      tc_fence_before();
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
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ BwdParams p) {
  using Geo = QueryGeom<HD>;
  constexpr uint32_t NS = Geo::NS;
  extern __shared__ uint8_t smem_raw[];
  float* sDel = reinterpret_cast<float*>(smem_raw);                  // [2][128] halves of Delta
  Item* items = reinterpret_cast<Item*>(sDel + 256);                 // [ITEMS]
  uint64_t* item_full = reinterpret_cast<uint64_t*>(items + ITEMS);  // [ITEMS]
  uint64_t* item_empty = item_full + ITEMS;  // [ITEMS]
  uint64_t* a_full = item_empty + ITEMS;     // Q and dO rows stored in TMEM, their stage read (8)
  uint64_t* del_full = a_full + 1;           // both halves of Delta stored (8 warps)
  uint64_t* full = del_full + 1;             // [NS] stage landed
  uint64_t* empty = full + NS;               // [NS] stage consumed
  uint64_t* s_full = empty + NS;             // S in TMEM
  uint64_t* dp_full = s_full + 1;            // dP in TMEM
  uint64_t* s_free = dp_full + 1;            // S read by the element-wise warps (8)
  uint64_t* ds_full = s_free + 1;            // dS stored (8 warps)
  uint64_t* acc_done = ds_full + 1;          // the item's dQ complete
  uint64_t* tail_ok = acc_done + 1;          // [2] the last K and V tiles are cleared behind the
                                             // sequence (in turn, as in the forward)
  uint64_t* drain = tail_ok + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t tiles_off = tiles_offset(smem_raw, Geo::SMALL, Geo::TILES_OFF);
  if (tiles_off == 0) {  // uniform
    if (threadIdx.x == 0) record_error(p.status, kStatusUnsupported, SITE_SMEM_LAYOUT);
    return;
  }
  uint8_t* sStage = smem_raw + tiles_off;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ITEMS; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], Geo::READERS);
    }
    mbar_init(a_full, 8);
    mbar_init(del_full, 8);
    for (uint32_t s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(s_free, 8);
    mbar_init(ds_full, 8);
    mbar_init(acc_done, 1);
    mbar_init(&tail_ok[0], 1);
    mbar_init(&tail_ok[1], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmDO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  uint32_t tmem = 0;
  if (warp == 0) {
    __syncwarp();
    start_arrive<Geo::THREADS>();
  } else {
    if (warp == 1) {
      tmem_alloc(tmem_slot, TMEM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    start_sync<Geo::THREADS>();
    tc_fence_after();
    tmem = *tmem_slot;
  }
  WaitBound wb{p.status, p.limit_ns, abort_flag};
  auto tiles_of = [&](const Item& it) { return (min(it.len, it.q0 + p.TPT) - 1) / TILE + 1; };
  // The stages are one ring of uses x = 0, 1, ...: an item's own rows, then its key tiles.

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    Item next{};
    Walk walk;
    prior_kernel_done();  // the lists, where there are any
    walk.next(p.src, next);
    const uint32_t box_rows = (uint32_t)(Geo::BOXES * 128) * (uint32_t)p.RU;
    bool ok = true;
    uint32_t n_items = 0, x = 0, n_tail = 0;  // items, stage uses and ragged items so far
    while (ok) {
      const Item it = next;
      const int slot = (int)(n_items % ITEMS);
      const int n = tiles_of(it);
      if (lane == 0) {
        ok = mbar_wait(&item_empty[slot], ((n_items / ITEMS) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
        if (ok) {
          items[slot] = it;
          mbar_arrive(&item_full[slot]);
        }
        for (int j = -1; ok && it.head >= 0 && j < n; ++j, ++x) {
          const uint32_t st = x % NS;
          ok = mbar_wait(&empty[st], ((x / NS) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
          if (!ok) break;
          uint8_t* a = sStage + st * Geo::STAGE;
          mbar_arrive_expect_tx(&full[st], j < 0 ? 2 * box_rows : 2 * Geo::TILE_B);
#pragma unroll
          for (int b = 0; b < Geo::BOXES; ++b) {
            if (j < 0) {
              tma_load_3d(a + b * BOX_BYTES, &tmQ, &full[st], 64 * b, it.head * p.G, it.start + it.q0);
              tma_load_3d(a + Geo::TILE_B + b * BOX_BYTES, &tmDO, &full[st], 64 * b, it.head * p.G,
                          it.start + it.q0);
            } else {
              tma_load_2d(a + b * BOX_BYTES, &tmK, &full[st], it.head * HD + 64 * b, it.start + j * TILE);
              tma_load_2d(a + Geo::TILE_B + b * BOX_BYTES, &tmV, &full[st], it.head * HD + 64 * b,
                          it.start + j * TILE);
            }
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      x = __shfl_sync(0xffffffffu, x, 0);
      if (!ok || it.head < 0) break;
      ++n_items;
      walk.next(p.src, next);
      if (n * TILE > it.len) {
        const uint32_t last = x - 1;
        // every lane reads the phase itself: the tiles are then visible to its writes
        ok = __all_sync(0xffffffffu, mbar_wait(&full[last % NS], (last / NS) & 1u, wb,
                                               SITE_PACKED_PRODUCER)) != 0;
        if (!ok) break;
        // K, then V
        clear_rows(sStage + (last % NS) * Geo::STAGE, 2 * Geo::BOXES, it.len - (n - 1) * TILE, lane, 32);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail_ok[n_tail & 1u]);
        ++n_tail;
      }
    }
    // the key side may take this multiprocessor over: its list is there, and all that it reads
    // but Delta (from the start on it would compete with the loads here: 402 against 399 us)
    dependents_may_start();
    if (lane == 0) {
      walk.end(p.src);
      // copies in flight land before the CTA ends
      WaitBound wd{p.status, p.limit_ns, nullptr};
      for (uint32_t b = x > NS ? x - NS : 0; b < x; ++b)
        mbar_wait(&full[b % NS], (b / NS) & 1u, wd, SITE_DRAIN);
      if (!ok) let_copies_land();
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
      auto issue_s = [&](uint32_t st) {
        const uint32_t k_lo = st_lo + st * (Geo::STAGE / 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ts_w(tmem + TM_SC, tmem + Geo::TM_Q + (uint32_t)(kk * 8), k_lo + kmajor_step(kk), st_hi,
                   idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(s_full);
      };
      auto issue_dp = [&](uint32_t st) {
        const uint32_t v_lo = st_lo + st * (Geo::STAGE / 16) + Geo::TILE_B / 16;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ts_w(tmem + TM_DP, tmem + Geo::TM_DO + (uint32_t)(kk * 8), v_lo + kmajor_step(kk), st_hi,
                   idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(dp_full);
      };
      auto issue_dq = [&](uint32_t st, bool first) {
        const uint32_t k_lo = mn_lo + st * (Geo::STAGE / 16);
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          mma_ts_w(tmem + 0, packed_step(tmem + TM_DP, kk), k_lo + (uint32_t)(kk * 128), mn_hi, idesc_acc,
                   (first && kk == 0) ? 0u : 1u);
        mma_commit(&empty[st]);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_poll(bar, parity & 1u, wb, SITE_PACKED_MMA);
      };
      bool ok = true;
      uint32_t n_items = 0, c = 0, n_tail = 0;  // items, key tiles, ragged items
      uint32_t st = 0, ph = 0;                  // the ring's next stage, and bit st: its phase
      while (ok) {
        const int slot = (int)(n_items % ITEMS);
        ok = wait(&item_full[slot], n_items / ITEMS);
        if (!ok) break;
        const Item it = items[slot];
        mbar_arrive(&item_empty[slot]);
        if (it.head < 0) break;
        const int n = tiles_of(it);
        const bool ragged = n * TILE > it.len;
        // the key tile of a stage is in place (cleared behind the sequence, if it is the last)
        auto wait_kv = [&](uint32_t at, bool last) {
          if (!wait(&full[at], ph >> at)) return false;
          ph ^= 1u << at;
          if (!ragged || !last) return true;
          const uint32_t turn = n_tail++;
          return wait(&tail_ok[turn & 1u], turn >> 1);
        };
        auto after = [](uint32_t at) { return at + 1 == NS ? 0u : at + 1; };
        // the own rows are in TMEM: their stage is free
        ok = wait(a_full, n_items);
        if (!ok) break;
        mbar_arrive(&empty[st]);
        ph ^= 1u << st;
        st = after(st);
        // S over the last tile's S of the item before, once that is in registers
        ok = wait_kv(st, n == 1) && (c == 0 || wait(s_free, c - 1));
        if (!ok) break;
        tc_fence_after();
        issue_s(st);
        issue_dp(st);
        for (int j = 0; j < n; ++j, ++c) {
          const bool more = j + 1 < n;
          const uint32_t then = after(st);
          if (more) {
            // next scores as soon as the element-wise warps hold this tile's
            ok = wait_kv(then, j + 2 == n) && wait(s_free, c);
            if (!ok) break;
            tc_fence_after();
            issue_s(then);
          }
          ok = wait(ds_full, c);
          if (!ok) break;
          tc_fence_after();
          issue_dq(st, j == 0);
          if (more) issue_dp(then);
          st = then;
        }
        if (ok) mma_commit(acc_done);
        ++n_items;
      }
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
    const uint32_t lane_base = tmem + ((uint32_t)(qq * 32) << 16);
    const uint32_t s_t = lane_base + TM_SC + (uint32_t)(g * GCOLS);
    const uint32_t d_t = lane_base + TM_DP + (uint32_t)(g * GCOLS);
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      const bool mine = mbar_wait(bar, parity & 1u, wb, SITE_PACKED_SOFTMAX);
      return __all_sync(0xffffffffu, mine) != 0;
    };
    // this thread's row in an item
    struct Row {
      int n;     // key tiles of the item; 0: no item is left
      int pos;   // position in the sequence, -1: no query
      int qh;    // query head
      long long row;
      float lse;
    };
    // 16-byte pieces of o per lane: half a row, but of the four rows of its group of lanes
    // the pieces 4 s + lane % 4, so that four lanes read 64 contiguous bytes
    constexpr int OW = HD / 16;
    const int quad = (lane & ~3) + qq * 32;  // the group's first row in the tile
    uint32_t n_items = 0, c = 0, x = 0;  // items, key tiles, stage uses
    // Takes the next item: its Q (warpgroup 0) or dO (warpgroup 1) row into TMEM, two bf16
    // values per column, as A operands; and this thread's pieces of o on the way to registers
    // (o[4 s + k]: piece 4 s + lane % 4 of the half row g of row quad + k), the same pieces of
    // dO in registers. The item's Q and dO columns are free: the products of the item before that
    // read them are complete (dP of its last tile was). Chunk w of row r lies at chunk
    // w ^ (r % 8) of its 128 bytes in shared memory (the 128-byte swizzle).
    auto take = [&](Row& r, uint4 (&o)[OW], uint4 (&d)[OW]) {
      r.n = 0;
      const int slot = (int)(n_items % ITEMS);
      if (!warp_wait(&item_full[slot], n_items / ITEMS)) return false;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      if (it.head < 0) return true;
      const bool row_ok = r_local < p.RU && it.q0 + tok < it.len;
      r.n = tiles_of(it);
      r.pos = row_ok ? it.q0 + tok : -1;
      r.qh = row_ok ? it.head * p.G + (r_local - tok * p.G) : 0;
      r.row = (long long)it.start + (row_ok ? r.pos : 0);
      r.lse = row_ok ? p.lse[(long long)r.qh * p.ld_lse + r.row] : INFINITY;
      if (r.n > 1) {
        const __nv_bfloat16* mine = row_ok ? p.o + r.row * p.ld_o + (long long)r.qh * HD + g * (HD / 2) : nullptr;
        __nv_bfloat16* rows[4];
        group_rows(const_cast<__nv_bfloat16*>(mine), rows);
#pragma unroll
        for (int w = 0; w < OW; ++w) {
          const uint4* from = reinterpret_cast<const uint4*>(rows[w & 3]) + (w & ~3) + (lane & 3);
          o[w] = rows[w & 3] != nullptr ? __ldg(from) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (!warp_wait(&full[x % NS], x / NS)) return false;
      const uint8_t* sQ = sStage + (x % NS) * Geo::STAGE;
      const uint8_t* sDO = sQ + Geo::TILE_B;
      x += 1 + r.n;
      const uint32_t dst = lane_base + (g == 0 ? Geo::TM_Q : Geo::TM_DO);
      const uint4* src = reinterpret_cast<const uint4*>((g == 0 ? sQ : sDO) + r_local * 128);
#pragma unroll
      for (int b = 0; b < Geo::BOXES; ++b) {
        uint32_t u[32];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const uint4 v = row_ok ? src[b * (BOX_BYTES / 16) + (w ^ (r_local & 7))] : make_uint4(0u, 0u, 0u, 0u);
          u[4 * w + 0] = v.x;
          u[4 * w + 1] = v.y;
          u[4 * w + 2] = v.z;
          u[4 * w + 3] = v.w;
        }
        tmem_st32(dst + (uint32_t)(32 * b), u);
      }
      if (r.n > 1) {
#pragma unroll
        for (int w = 0; w < OW; ++w) {
          const int row = quad + (w & 3);
          const int piece = g * OW + (w & ~3) + (lane & 3);  // of the row's HD / 8
          d[w] = *reinterpret_cast<const uint4*>(sDO + (piece >> 3) * BOX_BYTES + row * 128 +
                                                 16 * ((piece & 7) ^ (row & 7)));
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full);
      return true;
    };
    // This thread's half of Delta from o and dO, where there is more than one key tile.
    auto half_delta = [&](const Row& r, const uint4 (&o)[OW], const uint4 (&d)[OW]) {
      if (r.n <= 1) return;
      float part[4] = {0.f, 0.f, 0.f, 0.f};  // of rows quad + k
#pragma unroll
      for (int w = 0; w < OW; ++w) {
        const uint32_t a[4] = {o[w].x, o[w].y, o[w].z, o[w].w}, b[4] = {d[w].x, d[w].y, d[w].z, d[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          part[w & 3] = fmaf(bf16_lo(a[e]), bf16_lo(b[e]), part[w & 3]);
          part[w & 3] = fmaf(bf16_hi(a[e]), bf16_hi(b[e]), part[w & 3]);
        }
      }
      float del = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        part[k] += __shfl_xor_sync(0xffffffffu, part[k], 1);
        part[k] += __shfl_xor_sync(0xffffffffu, part[k], 2);
        if ((lane & 3) == k) del = part[k];
      }
      sDel[g * 128 + r_local] = r.pos < 0 ? 0.f : del;
      __syncwarp();
      if (lane == 0) mbar_arrive(del_full);
    };
    // the short sequences, under the first item's loads
    prior_kernel_done();  // the lists, where there are any
    short_query_side<HD>(p, (gridDim.x - 1u - blockIdx.x) * 8u + (unsigned)(warp - 2), gridDim.x * 8u);
    Row cur;
    bool ok;
    {
      uint4 o[OW], d[OW];
      ok = take(cur, o, d);
      if (ok) half_delta(cur, o, d);
    }
    while (ok && cur.n > 0) {
      float del = 0.f;
      for (int j = 0; j < cur.n; ++j, ++c) {
        if (!warp_wait(s_full, c)) {
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
          for (int e = 0; e < 32; ++e) {
            pf[e] = ex2(fmaf(__uint_as_float(s0[e]), p.scale_log2, -cur.lse));
            pf[32 + e] = ex2(fmaf(__uint_as_float(s1[e]), p.scale_log2, -cur.lse));
          }
        }
        const int kbase = j * TILE + g * GCOLS;
        // some key of the group is in the row's future
        const bool masked = kbase + GCOLS - 1 > cur.pos;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 64; ++e) pf[e] = kbase + e <= cur.pos ? pf[e] : 0.f;
        }
        // ---- dS = P (dP - Delta)
        if (!warp_wait(dp_full, c)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (cur.n == 1) {
          // one tile holds all keys: Delta from P and dP themselves. There o is a mean of few
          // values, and its rounding would be the largest error of dS.
          float part = 0.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t gv[32];
            tmem_ld32(d_t + (uint32_t)(32 * half), gv);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (kbase + 32 * half + e <= cur.pos)
                part = fmaf(pf[32 * half + e], __uint_as_float(gv[e]), part);
          }
          sDel[g * 128 + r_local] = part;
          __syncwarp();
          if (lane == 0) mbar_arrive(del_full);
        }
        if (j == 0) {
          if (!warp_wait(del_full, n_items)) {
            ok = false;
            break;
          }
          del = sDel[r_local] + sDel[128 + r_local];
          if (g == 1 && cur.pos >= 0) p.delta[(long long)cur.qh * p.ld_delta + cur.row] = del;
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
              if (kbase + 32 * half + e > cur.pos) gv[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int at = 32 * half + e;
            float d0, d1;
            f2_unpack(f2_mul(f2_pack(pf[at], pf[at + 1]),
                             f2_sub(f2_pack(__uint_as_float(gv[e]), __uint_as_float(gv[e + 1])), del2)),
                      d0, d1);
            dd[at >> 1] = pack_bf16x2(d0, d1);
          }
        }
        tmem_st32(d_t, dd);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      // the next item's rows go to TMEM before this one's epilogue, so that its first
      // products run under it; its first dQ waits for the dS that comes after the epilogue
      const uint32_t done = n_items++;
      Row nxt;
      uint4 o[OW], d[OW];
      ok = take(nxt, o, d);
      if (!ok || !warp_wait(acc_done, done)) break;
      // ---------------------------------------------------------- epilogue
      tc_fence_after();
      __nv_bfloat16* dst[4];
      group_rows(cur.pos >= 0 ? p.dq + cur.row * p.ld_dq + (long long)cur.qh * HD + g * (HD / 2) : nullptr, dst);
#pragma unroll
      for (int e0 = 0; e0 < HD / 2; e0 += 32) {
        uint32_t a[32], w[16];
        tmem_ld32(lane_base + (uint32_t)(g * (HD / 2) + e0), a);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack_bf16x2(__uint_as_float(a[2 * e]) * p.scale, __uint_as_float(a[2 * e + 1]) * p.scale);
        store_rows(w, dst);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (dst[k] != nullptr) dst[k] += 32;
      }
      tc_fence_before();
      half_delta(nxt, o, d);
      cur = nxt;
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
                      const void* q, int64_t ld_q, const void* dout, int64_t ld_do, const void* k,
                      int64_t ld_k, const void* v, int64_t ld_v, cudaStream_t stream) {
  CUtensorMap tq, tdo, tk, tv;
  TSP_TRY(make_query_map(&tq, s, q, ld_q));
  TSP_TRY(make_query_map(&tdo, s, dout, ld_do));
  const uint64_t cols = (uint64_t)s.kv_heads * HD, rows = (uint64_t)s.tokens;
  TSP_TRY(make_tmap_2d_bf16(&tk, k, cols, rows, (uint64_t)ld_k * 2, 64, TILE));
  TSP_TRY(make_tmap_2d_bf16(&tv, v, cols, rows, (uint64_t)ld_v * 2, 64, TILE));
  {
    auto kernel = packed_bwd_dq_kernel<HD>;
    const size_t smem = QueryGeom<HD>::SMEM;
    TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                              "packed attention backward: cudaFuncSetAttribute"));
    p.src = queries;
    const unsigned grid = (unsigned)std::min<long long>((long long)queries.max_items * s.kv_heads, sm_count());
    cudaError_t e;
    if (p.src.items != nullptr) {  // behind the kernel that writes the lists
      e = launch_early(kernel, grid, QueryGeom<HD>::THREADS, smem, stream, tq, tdo, tk, tv, p);
    } else {
      kernel<<<grid, QueryGeom<HD>::THREADS, smem, stream>>>(tq, tdo, tk, tv, p);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return cuda_fail(e, "packed attention backward (query side): launch");
  }
  {
    auto kernel = packed_bwd_dkv_kernel<HD>;
    const size_t smem = KeyGeom<HD>::SMEM;
    TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                              "packed attention backward: cudaFuncSetAttribute"));
    p.src = keys;
    const unsigned grid = (unsigned)std::min<long long>((long long)keys.max_items * s.kv_heads, sm_count());
    cudaError_t e = launch_early(kernel, grid, KeyGeom<HD>::THREADS, smem, stream, tq, tdo, tk, tv, p);
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
  TSP_GUARD_BEGIN
  const char* what = "tsp_packed_attention_bwd";
  Shape s;
  TSP_TRY(make_shape(what, tokens, n_seqs, heads, kv_heads, head_dim, &s));
  TSP_TRY(check_scale(what, scale));
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
  p.o = in(o);
  p.ld_o = ld_o;
  p.q = in(q);
  p.k = in(k);
  p.v = in(v);
  p.dout = in(dout);
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_v = ld_v;
  p.ld_do = ld_do;
  p.lse = lse;
  p.ld_lse = ld_lse;
  p.delta = at<float>(ws, w.delta);
  p.ld_delta = w.ld_stat;
  p.G = s.G;
  p.TPT = s.TPT;
  p.RU = s.RU;
  p.scale_log2 = LOG2E * scale;
  p.scale = scale;
  p.status = status_of(ws);
  p.limit_ns = wait_limit_ns();
  int* counts = at<int>(ws, w.counts);
  // 48 MB of K and V in L2 at a time, as for the plan's backward
  const int group = head_group(s, 48ll << 20);
  Source queries = make_source(s, starts, s.TPT, false, group, at<Item>(ws, w.items), counts,
                               (int)w.max_query, ws, 1);
  Source keys = make_source(s, starts, TILE, true, group, at<Item>(ws, w.key_items), counts + 1,
                            (int)w.max_key, ws, 2);
  if (queries.items != nullptr) {
    queries.short_last = keys.short_last = queries.items + w.max_query - 1;
    queries.short_count = keys.short_count = counts + 2;
    const ListArgs a{s.TPT, 0, list_shift((tokens + TILE - 1) / TILE), at<Item>(ws, w.items), counts,
                     (int)w.max_query};
    const ListArgs b{TILE, s.TPT, list_shift((tokens + s.TPT - 1) / s.TPT), at<Item>(ws, w.key_items),
                     counts + 1, (int)w.max_key};
    TSP_TRY(launch_lists(s, starts, a, b, counts + 2, p.status, st));
  }
  if (head_dim == 64) return launch_bwd<64>(s, queries, keys, p, q, ld_q, dout, ld_do, k, ld_k, v, ld_v, st);
  return launch_bwd<128>(s, queries, keys, p, q, ld_q, dout, ld_do, k, ld_k, v, ld_v, st);
  TSP_GUARD_END
}
