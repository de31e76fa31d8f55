// packed_attention.cu - causal attention over a packed batch with grouped query heads.
//
// Sequences of any lengths lie back to back on one token axis: sequence s owns rows
// [starts[s], starts[s+1]). Query head h reads key head h / G, G = heads / kv_heads. For
// the token at position i of its sequence
//     o_i = sum_{j <= i} exp(scale q_i.k_j - m_i) v_j / l_i
// over the keys of its own sequence only; lse_i = log2 of the sum of exp(scale q_i.k_j).
// Bound: the tensor cores (4 d operations per visible pair and head) from a few thousand
// tokens per sequence on; launch and fill latency for a handful of short prompts.
//
// A query tile is 128 rows of TPT = floor(128 / G) tokens times the G heads that share a
// key head (row = token * G + head; one TMA box of 64 columns x G heads x TPT tokens lays
// them out), so a K/V tile serves the whole group, and a short sequence fills G times more
// of its tile than one head alone would. Tiles never span sequences: a sequence's result
// has the same bits whatever else is packed beside it. Sequences of a few tokens go to no
// tile: the softmax warps take them first, on the CUDA cores (packed_short.cuh).
//
// A CTA works on two neighbouring query tiles (A and B) of one key head, its item:
//   warp 0      finds the items, and loads by TMA: Q_A, Q_B, K_0, then pairs (V_j, K_{j+1})
//               into a 2-stage ring; then clears what follows the sequence in its last V tile
//   warp 1      TMEM allocation; one lane issues per key tile O_A += P_A V_j,
//               S_A = Q_A K_{j+1}^T, and the same for B: while one tile's softmax runs,
//               the tensor core works for the other
//   warps 2..5  softmax and epilogue of tile A, warps 6..9 of tile B, one row per thread:
//               online softmax in base 2 with a running maximum that only moves when it is
//               exceeded by more than 8 (P <= 256; O and l are rescaled then), P written
//               as bf16 over the scores' TMEM columns as the A operand of P V
// TMEM columns: S_A [0,128) O_A [128,256) S_B [256,384) O_B [384,512).
// P is rounded to bf16 for the tensor core while l sums the fp32 values: at most 2^-8 of a
// term, and the terms' errors cancel in the sum where o's own rounding does not.
//
// CTAs are persistent, one per multiprocessor, and the roles meet only at barriers whose
// phases run on across items: the next item's loads and first scores are under way while the
// last one is stored. Items are (sequence, tile pair) sorted by their number of key tiles,
// longest first, and drawn from a counter. Up to 128 sequences warp 0 finds an item in
// `starts` by a search in registers; beyond, a small kernel writes the sorted list first.
// starts is data, not a launch parameter: a captured graph may be replayed with other
// lengths. Starts that decrease or leave the buffers give no items and an error in the
// status word.
//
// A key tile at a sequence's end reads on into the next sequence, or into rows that belong
// to none. Their scores are replaced by -inf, so P is 0 there, but 0 times a NaN or an
// infinity in V is not 0: warp 0 overwrites those rows of V with zeros in shared memory
// before the product may start.
//
// Measured, 32 query and 8 key heads of 128: one sequence of 32768 tokens and 1000 others 6.0 to
// 6.2 ms, 1425 to 1460 TFLOP/s (0.75 of the measured burst rate); 16384 tokens in 18 sequences
// 0.39 ms, 1220 TFLOP/s, against 0.42 with a CTA per item and 0.40 with rows stored lane by lane;
// 128 sequences of 128 tokens 0.08 ms (0.05 of it HBM). What binds the long sequence is the latency
// of a tile's chain (scores, their load from tensor memory, softmax, P, product) through two tiles
// in turn: the schedulers issue 0.36 instructions a cycle, the exponential unit is 32% busy, the
// tensor pipe 63% (55% in the ragged batch), and 3.5 warps per issue wait for a load.
#include <algorithm>
#include <cmath>

#include "attention_math.cuh"
#include "packed_attention.cuh"
#include "packed_short.cuh"

namespace tsp {
namespace packed {
namespace {

constexpr int QT = TILE, KT = TILE;
constexpr int STAGES = 2;
constexpr int THREADS = 320;
constexpr uint32_t TMEM_COLS = 512;
constexpr int ITEMS = 4;  // items between the producer and the epilogue
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units

__device__ __forceinline__ uint32_t tm_s(int t) { return t ? 256u : 0u; }
__device__ __forceinline__ uint32_t tm_o(int t) { return t ? 384u : 128u; }

// ------------------------------------------------------------------ work lists
constexpr int LIST_THREADS = 1024;

// f(any, start, len, first token) for every item, by whole warps (lanes with `any` false have
// none): a thread fetches one sequence and takes it if it is a single item; of the others, a
// warp walks one sequence after the other, lane by lane over its items.
template <class F>
__device__ __forceinline__ void each_item(const int32_t* starts, int n, int tile, int short_len, F f) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < n; base += LIST_THREADS) {
    const int i = base + threadIdx.x;
    const int start = i < n ? starts[i] : 0, len = i < n ? starts[i + 1] - start : 0;
    f(len > short_len && len <= tile, start, len, 0);
    for (unsigned left = __ballot_sync(0xffffffffu, len > short_len && len > tile); left; left &= left - 1) {
      const int from = __ffs(left) - 1;
      const int s = __shfl_sync(0xffffffffu, start, from);
      const int m = __shfl_sync(0xffffffffu, len, from);
      for (long long q0 = 0; q0 < m; q0 += 32ll * tile) {
        const long long mine = q0 + (long long)lane * tile;
        f(mine < m, s, m, (int)mine);
      }
    }
  }
}

// Adds one to counter[b] for every lane with `any` and returns the lane's own number, with one
// atomic per distinct b of the warp: most items of a batch of short sequences cost the same.
__device__ __forceinline__ int claim(int* counter, int b, bool any) {
  const unsigned active = __ballot_sync(0xffffffffu, any);
  if (!any) return -1;
  const int lane = threadIdx.x & 31;
  const unsigned peers = __match_any_sync(active, b);
  const int leader = __ffs(peers) - 1;
  int first = 0;
  if (lane == leader) first = atomicAdd(&counter[b], __popc(peers));
  return __shfl_sync(peers, first, leader) + __popc(peers & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(LIST_THREADS)
    packed_lists_kernel(const int32_t* __restrict__ starts, int n, long long tokens, ListArgs a,
                        ListArgs b, int short_len, int* short_count, DevStatus* status) {
  dependents_may_start();
  const ListArgs l = blockIdx.x == 0 ? a : b;
  __shared__ int hist[1024];
  __shared__ int sums[32];
  __shared__ int n_short;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  hist[tid] = 0;
  if (tid == 0) n_short = 0;
  bool ok = true;
  for (int i = tid; i < n; i += LIST_THREADS)
    ok = ok && starts[i] >= 0 && starts[i + 1] >= starts[i] && starts[i + 1] <= tokens;
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      *l.count = 0;
      if (blockIdx.x == 0) *short_count = 0;
      record_error(status, kStatusInvalid, SITE_PACKED_STARTS);
    }
    return;
  }
  auto bucket = [&](int len, int q0) {
    const int cost = l.streamed ? (len - 1) / l.streamed - q0 / l.streamed
                                : (min((long long)len, (long long)q0 + l.tile) - 1) / TILE;
    return min(cost >> l.shift, 1023);
  };
  each_item(starts, n, l.tile, short_len, [&](bool any, int, int len, int q0) {
    claim(hist, any ? bucket(len, q0) : 0, any);
  });
  __syncthreads();
  // first slot of each bucket, the costliest bucket first
  const int mine = hist[1023 - tid];
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    sums[lane] = v;
  }
  __syncthreads();
  incl += warp ? sums[warp - 1] : 0;
  hist[1023 - tid] = incl - mine;
  if (tid == LIST_THREADS - 1) *l.count = min(incl, l.max_items);
  __syncthreads();
  // the order inside a bucket may change from run to run: every item is its own CTA's work
  each_item(starts, n, l.tile, short_len, [&](bool any, int s, int len, int q0) {
    const int slot = claim(hist, any ? bucket(len, q0) : 0, any);
    if (any && slot < l.max_items) l.items[slot] = Item{s, len, q0, 0};
  });
  if (blockIdx.x == 0) {
    // the short sequences, for every kernel behind this one: from the other end of the list,
    // which has a place for each, since a sequence that is short has no item
    for (int base = 0; base < n; base += LIST_THREADS) {
      const int i = base + tid;
      const int start = i < n ? starts[i] : 0, len = i < n ? starts[i + 1] - start : 0;
      const bool is = len > 0 && len <= short_len;
      const int slot = claim(&n_short, 0, is);
      if (is) l.items[l.max_items - 1 - slot] = Item{start, len, 0, 0};
    }
    __syncthreads();
    if (tid == 0) *short_count = n_short;
  }
}

// ------------------------------------------------------------------ forward
template <int HD>
struct Geometry {
  static constexpr int BOXES = HD / 64;
  static constexpr uint32_t TILE_BYTES = 128 * HD * 2;
  // Q_A, Q_B, K_0, then the ring: K slots 0/1 and V slots 0/1
  static constexpr size_t USED = 1024 + (size_t)(3 + 2 * STAGES) * TILE_BYTES + 512;
  // all 512 TMEM columns: alone on its SM
  static constexpr size_t SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
};

struct FwdParams {
  const __nv_bfloat16* q;  // read directly for the short sequences
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long ld_q, ld_k, ld_v;
  __nv_bfloat16* o;
  long long ld_o;
  float* lse;  // optional [heads][ld_lse]
  long long ld_lse;
  Source src;
  int G, TPT, RU;
  float scale_log2;
  DevStatus* status;
  unsigned long long limit_ns;
};

// Tiles of an item: key tiles of query tile A and of B (0: B has no query).
struct Tiles {
  int a, b, n;
  bool ragged;  // the last key tile reads on behind the sequence
};
__device__ __forceinline__ Tiles tiles_of(const Item& it, int tpt) {
  const int q_b = it.q0 + tpt;
  Tiles t;
  t.a = (min(it.len, q_b) + KT - 1) / KT;
  t.b = q_b < it.len ? (min(it.len, q_b + tpt) + KT - 1) / KT : 0;
  t.n = max(t.a, t.b);
  t.ragged = t.n * KT > it.len;
  return t;
}

template <int HD>
__global__ void __launch_bounds__(THREADS, 1)
    packed_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                            const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const FwdParams p) {
  using Geo = Geometry<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK0 = sQ + 2 * Geo::TILE_BYTES;
  uint8_t* sK = sK0 + Geo::TILE_BYTES;
  uint8_t* sV = sK + STAGES * Geo::TILE_BYTES;
  Item* items = reinterpret_cast<Item*>(sV + STAGES * Geo::TILE_BYTES);  // [ITEMS]
  uint64_t* item_full = reinterpret_cast<uint64_t*>(items + ITEMS);      // [ITEMS]
  uint64_t* item_empty = item_full + ITEMS;  // [ITEMS] read by the MMA lane and 8 warps
  uint64_t* q_full = item_empty + ITEMS;     // Q_A, Q_B, K_0 of the item
  uint64_t* q_empty = q_full + 1;            // its scores are all computed
  uint64_t* kv_full = q_empty + 1;           // [STAGES] V_j and K_{j+1}
  uint64_t* kv_empty = kv_full + STAGES;     // [STAGES]
  uint64_t* s_full = kv_empty + STAGES;      // [2] per tile: S(j) in TMEM
  uint64_t* p_full = s_full + 2;             // [2] per tile: P(j) in TMEM (4 warps)
  uint64_t* o_done = p_full + 2;             // [2] per tile: the item's last O += P V complete
  // the last V tile is cleared behind the sequence: two in turn, because the producer may
  // clear the next item's before the MMA lane has waited for this one's
  uint64_t* tail_ok = o_done + 2;            // [2]
  uint64_t* drain = tail_ok + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ITEMS; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], 9);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(&tail_ok[0], 1);
    mbar_init(&tail_ok[1], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  uint32_t tmem = 0;
  if (warp == 0) {
    __syncwarp();
    start_arrive<THREADS>();
  } else {
    if (warp == 1) {
      tmem_alloc(tmem_slot, TMEM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    start_sync<THREADS>();
    tc_fence_after();
    tmem = *tmem_slot;
  }
  WaitBound wb{p.status, p.limit_ns, abort_flag};

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    WaitBound wd{p.status, p.limit_ns, nullptr};
    Item next{};
    Walk walk;
    prior_kernel_done();  // the list, where there is one
    walk.next(p.src, next);
    bool ok = true;
    uint32_t n_items = 0, c = 0, n_tail = 0;  // items, key tiles and ragged items so far
    while (ok) {
      const Item it = next;
      const int slot = (int)(n_items % ITEMS);
      const Tiles tl = tiles_of(it, p.TPT);
      if (lane == 0) {
        ok = mbar_wait(&item_empty[slot], ((n_items / ITEMS) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
        if (ok) {
          items[slot] = it;
          mbar_arrive(&item_full[slot]);
        }
        if (ok && it.head >= 0) {
          ok = mbar_wait(q_empty, (n_items & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
          if (ok) {
            const uint32_t q_bytes = (uint32_t)(Geo::BOXES * 128) * (uint32_t)p.RU;
            mbar_arrive_expect_tx(q_full, (tl.b ? 2u : 1u) * q_bytes + Geo::TILE_BYTES);
#pragma unroll
            for (int b = 0; b < Geo::BOXES; ++b) {
              tma_load_3d(sQ + b * BOX_BYTES, &tmQ, q_full, 64 * b, it.head * p.G, it.start + it.q0);
              if (tl.b)
                tma_load_3d(sQ + Geo::TILE_BYTES + b * BOX_BYTES, &tmQ, q_full, 64 * b, it.head * p.G,
                            it.start + it.q0 + p.TPT);
              tma_load_2d(sK0 + b * BOX_BYTES, &tmK, q_full, it.head * HD + 64 * b, it.start);
            }
          }
          for (int j = 0; ok && j < tl.n; ++j, ++c) {
            const int st = (int)(c % STAGES);
            ok = mbar_wait(&kv_empty[st], ((c / STAGES) & 1u) ^ 1u, wb, SITE_PACKED_PRODUCER);
            if (!ok) break;
            const bool has_k = j + 1 < tl.n;
            mbar_arrive_expect_tx(&kv_full[st], (has_k ? 2u : 1u) * Geo::TILE_BYTES);
#pragma unroll
            for (int b = 0; b < Geo::BOXES; ++b) {
              tma_load_2d(sV + st * Geo::TILE_BYTES + b * BOX_BYTES, &tmV, &kv_full[st],
                          it.head * HD + 64 * b, it.start + j * KT);
              if (has_k)
                tma_load_2d(sK + st * Geo::TILE_BYTES + b * BOX_BYTES, &tmK, &kv_full[st],
                            it.head * HD + 64 * b, it.start + (j + 1) * KT);
            }
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      c = __shfl_sync(0xffffffffu, c, 0);
      if (!ok || it.head < 0) break;
      // the next item is looked up while the last loads are on their way
      walk.next(p.src, next);
      if (tl.ragged) {
        const uint32_t last = c - 1;
        const int st = (int)(last % STAGES);
        // every lane reads the phase itself: the tile is then visible to its writes
        ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[st], (last / STAGES) & 1u, wb,
                                               SITE_PACKED_PRODUCER)) != 0;
        if (!ok) break;
        const int keep = it.len - (tl.n - 1) * KT;  // rows of the sequence in the tile
#pragma unroll
        for (int b = 0; b < Geo::BOXES; ++b) {
          uint4* rows = reinterpret_cast<uint4*>(sV + st * Geo::TILE_BYTES + b * BOX_BYTES);
          for (int i = keep * 8 + lane; i < 128 * 8; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail_ok[n_tail & 1u]);
        ++n_tail;
      }
      ++n_items;
    }
    if (lane == 0) {
      walk.end(p.src);
      // copies in flight land before the CTA ends: the last use of each barrier that was armed
      // (after a wait that gave up, a millisecond for what its item may have left)
      if (n_items > 0) mbar_wait(q_full, (n_items - 1) & 1u, wd, SITE_DRAIN);
      for (uint32_t b = c > STAGES ? c - STAGES : 0; b < c; ++b)
        mbar_wait(&kv_full[b % STAGES], (b / STAGES) & 1u, wd, SITE_DRAIN);
      if (!ok) {
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 1000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc_s = make_idesc_bf16(QT, KT, false);
      const uint32_t idesc_o = make_idesc_bf16(QT, HD, true);
      const uint64_t dq0 = make_sdesc_sw128(smem_addr(sQ), 16, 1024);
      const uint64_t dk0 = make_sdesc_sw128(smem_addr(sK0), 16, 1024);
      const uint64_t dv0 = make_sdesc_sw128(smem_addr(sV), BOX_BYTES, 1024);
      const uint32_t q_hi = (uint32_t)(dq0 >> 32), k_hi = (uint32_t)(dk0 >> 32);
      const uint32_t v_hi = (uint32_t)(dv0 >> 32);
      constexpr uint32_t TILE16 = Geo::TILE_BYTES >> 4;
      // S_t = Q_t K^T with K in `slot` (0: the item's first key tile, 1 + stage otherwise)
      auto issue_s = [&](int t, uint32_t slot) {
        const uint32_t a_lo = (uint32_t)dq0 + (uint32_t)t * TILE16;
        const uint32_t b_lo = (uint32_t)dk0 + slot * TILE16;
        const uint32_t d = tmem + tm_s(t);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = (uint32_t)(((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4);
          mma_ss_w(d, a_lo + off, q_hi, b_lo + off, k_hi, idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[t]);
      };
      auto issue_pv = [&](int t, uint32_t stage, bool first) {
        const uint32_t b_lo = (uint32_t)dv0 + stage * TILE16;
        const uint32_t d = tmem + tm_o(t), a = tmem + tm_s(t);
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_ts_w(d, a + (uint32_t)(kk * 8), b_lo + (uint32_t)(kk * (2048 >> 4)), v_hi, idesc_o,
                   kk > 0 ? 1u : (first ? 0u : 1u));
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_poll(bar, parity & 1u, wb, SITE_PACKED_MMA);
      };
      bool ok = true;
      uint32_t n_items = 0, c = 0, n_tail = 0;
      uint32_t cp[2] = {0, 0};  // P tiles taken so far
      while (ok) {
        const int slot = (int)(n_items % ITEMS);
        ok = wait(&item_full[slot], n_items / ITEMS);
        if (!ok) break;
        const Item it = items[slot];
        mbar_arrive(&item_empty[slot]);
        if (it.head < 0) break;
        const Tiles tl = tiles_of(it, p.TPT);
        ok = wait(q_full, n_items);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, 0);
        if (tl.b > 0) issue_s(1, 0);
        if (tl.n == 1) mma_commit(q_empty);
        ok = wait(&kv_full[c % STAGES], c / STAGES);
        for (int j = 0; ok && j < tl.n; ++j, ++c) {
          const uint32_t st = c % STAGES;
          if (tl.ragged && j == tl.n - 1) {
            ok = wait(&tail_ok[n_tail & 1u], n_tail >> 1);
            ++n_tail;
            if (!ok) break;
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? tl.b : tl.a;
            if (ok && j < nt) {
              ok = wait(&p_full[t], cp[t]);
              ++cp[t];
              if (ok) {
                tc_fence_after();
                issue_pv(t, st, j == 0);
                if (j + 1 < nt) {
                  issue_s(t, 1 + st);
                } else {
                  mma_commit(&o_done[t]);
                }
              }
            }
            // while tile A's products run, wait for the next stage
            if (ok && t == 0 && j + 1 < tl.n) ok = wait(&kv_full[(c + 1) % STAGES], (c + 1) / STAGES);
          }
          if (!ok) break;
          mma_commit(&kv_empty[st]);
          if (j + 2 == tl.n) mma_commit(q_empty);  // the item's last scores are issued
        }
        ++n_items;
      }
      mma_commit(drain);
      WaitBound wd{p.status, p.limit_ns, nullptr};
      mbar_wait(drain, 0, wd, SITE_DRAIN);
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int t = (warp - 2) >> 2;
    const int q = warp & 3;
    const int r_local = q * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t s_tmem = lane_base + tm_s(t);
    const uint32_t o_tmem = lane_base + tm_o(t);
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      const WaitBound wbs{p.status, p.limit_ns, abort_flag};
      const bool mine = mbar_wait(bar, parity & 1u, wbs, SITE_PACKED_SOFTMAX);
      return __all_sync(0xffffffffu, mine) != 0;
    };
    // the short sequences, under the first item's loads; dealt out from the last CTA on, since
    // the last ones have the cheapest item or none
    prior_kernel_done();  // the list, where there is one
    short_forward<HD>(p, (gridDim.x - 1u - blockIdx.x) * 8u + (unsigned)(warp - 2), gridDim.x * 8u);
    uint32_t n_items = 0;
    uint32_t ph = 0;  // phase bits: 1 of s_full, 2 of o_done
    while (true) {
      const int slot = (int)(n_items % ITEMS);
      if (!warp_wait(&item_full[slot], n_items / ITEMS)) break;
      ++n_items;
      // what the epilogue needs of the item is read again there, instead of being held in
      // registers across the key loop; only then is the slot released
      int my_tiles, pos;
      {
        const Item it = items[slot];
        if (it.head < 0) break;
        const Tiles tl = tiles_of(it, p.TPT);
        const int at = it.q0 + (t ? p.TPT : 0) + r_local / p.G;
        my_tiles = t ? tl.b : tl.a;
        pos = r_local < p.RU && at < it.len ? at : -1;
      }
      if (my_tiles == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[slot]);
        continue;
      }
      float m_ref = -INFINITY;  // reference maximum (scaled, log2 units)
      float l = 0.f;
      bool ok = true;
      for (int j = 0; j < my_tiles; ++j, ph ^= 1u) {
        // S(j) complete also means O += P(j-1) V_{j-1} is complete (in-order MMAs)
        if (!warp_wait(&s_full[t], ph)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sc[KT];
        {
          uint32_t ra[32], rb[32], rc[32], rd[32];
          tmem_ld32(s_tmem + 0, ra);
          tmem_ld32(s_tmem + 32, rb);
          tmem_ld32(s_tmem + 64, rc);
          tmem_ld32(s_tmem + 96, rd);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            sc[e] = __uint_as_float(ra[e]);
            sc[32 + e] = __uint_as_float(rb[e]);
            sc[64 + e] = __uint_as_float(rc[e]);
            sc[96 + e] = __uint_as_float(rd[e]);
          }
        }
        const int kv0 = j * KT;
        if (kv0 + KT - 1 > pos) {
#pragma unroll
          for (int e = 0; e < KT; ++e)
            if (kv0 + e > pos) sc[e] = -INFINITY;
        }
        float m4[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
        for (int e = 4; e + 8 <= KT; e += 8) {
#pragma unroll
          for (int u = 0; u < 4; ++u) m4[u] = max3f(m4[u], sc[e + u], sc[e + 4 + u]);
        }
        const float mraw = max3f(max3f(m4[0], m4[1], sc[KT - 4]), max3f(m4[2], m4[3], sc[KT - 3]),
                                 fmaxf(sc[KT - 2], sc[KT - 1]));
        const float mx = mraw * p.scale_log2;  // scale > 0 keeps the order
        float factor = 1.f;
        const bool rescale = mx > m_ref + RESCALE_THRESHOLD;
        if (rescale) {
          factor = ex2(m_ref - mx);  // 0 when m_ref is still -inf
          m_ref = mx;
        }
        const float neg_ref = m_ref == -INFINITY ? 0.f : -m_ref;
        l *= factor;
        l += exp_tile<KT>(sc, s_tmem, p.scale_log2, neg_ref);
        // rescale O before P(j) is handed over; after the exponentials, when the scores are
        // no longer live
        if (j > 0 && __any_sync(0xffffffffu, rescale && factor != 1.f)) {
#pragma unroll 1
          for (int e0 = 0; e0 < HD; e0 += 16) {
            uint32_t r[16];
            tmem_ld16(o_tmem + e0, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * factor);
            tmem_st16(o_tmem + e0, r);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok || !warp_wait(&o_done[t], ph >> 1)) break;
      ph ^= 2u;
      // ---------------------------------------------------------- epilogue
      // P of the next item is handed over after these loads, and only then may its first
      // product overwrite O
      tc_fence_after();
      const bool row_ok = pos >= 0;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      const int tok = r_local / p.G;
      const long long row = (long long)it.start + (row_ok ? pos : 0);
      const int qh = it.head * p.G + (r_local - tok * p.G);
      const float inv = 1.f / l;
      if (p.lse != nullptr && row_ok) p.lse[(long long)qh * p.ld_lse + row] = m_ref + log2f(l);
      __nv_bfloat16* dst[4];
      group_rows(row_ok ? p.o + row * p.ld_o + (long long)qh * HD : nullptr, dst);
#pragma unroll
      for (int e0 = 0; e0 < HD; e0 += 32) {
        uint32_t r[32], w[16];
        tmem_ld32(o_tmem + e0, r);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
        store_rows(w, dst);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (dst[k] != nullptr) dst[k] += 32;
      }
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

template <int HD>
tsp_status launch_fwd(const Shape& s, const FwdParams& p, const void* q, int64_t ld_q, const void* k,
                      int64_t ld_k, const void* v, int64_t ld_v, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  TSP_TRY(make_query_map(&tq, s, q, ld_q));
  const uint64_t cols = (uint64_t)s.kv_heads * HD, rows = (uint64_t)s.tokens;
  TSP_TRY(make_tmap_2d_bf16(&tk, k, cols, rows, (uint64_t)ld_k * 2, 64, KT));
  TSP_TRY(make_tmap_2d_bf16(&tv, v, cols, rows, (uint64_t)ld_v * 2, 64, KT));
  auto kernel = packed_attention_kernel<HD>;
  const size_t smem = Geometry<HD>::SMEM;
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                            "packed attention: cudaFuncSetAttribute"));
  const unsigned grid = (unsigned)std::min<long long>((long long)p.src.max_items * s.kv_heads, sm_count());
  cudaError_t e;
  if (p.src.items != nullptr) {  // behind the kernel that writes the list
    e = launch_early(kernel, grid, THREADS, smem, stream, tq, tk, tv, p);
  } else {
    kernel<<<grid, THREADS, smem, stream>>>(tq, tk, tv, p);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "packed attention: launch");
}

}  // namespace

tsp_status make_shape(const char* what, int64_t tokens, int n_seqs, int heads, int kv_heads,
                      int head_dim, Shape* s) {
  const std::string w(what);
  if (tokens < 0 || tokens > (1ll << 30) || n_seqs < 0 || n_seqs > (1 << 20))
    return fail(TSP_ERR_UNSUPPORTED, w + ": tokens in [0, 2^30] and sequences in [0, 2^20] only");
  if (head_dim != 64 && head_dim != 128)
    return fail(TSP_ERR_UNSUPPORTED, w + ": head_dim 64 or 128");
  if (heads < 1 || kv_heads < 1 || heads % kv_heads || heads / kv_heads > TILE || heads > 65536)
    return fail(TSP_ERR_UNSUPPORTED,
                w + ": heads must be 1 to 128 times kv_heads, and at most 65536");
  s->tokens = tokens;
  s->n_seqs = n_seqs;
  s->heads = heads;
  s->kv_heads = kv_heads;
  s->d = head_dim;
  s->G = heads / kv_heads;
  s->TPT = TILE / s->G;
  s->RU = s->TPT * s->G;
  // one CTA per query tile and key head at most, as the backward launches them
  if ((tokens / s->TPT + n_seqs + tokens / TILE) * (int64_t)kv_heads > (1ll << 31) - 1)
    return fail(TSP_ERR_UNSUPPORTED, w + ": too many tiles for one launch");
  return TSP_OK;
}

Workspace make_workspace(const Shape& s) {
  Workspace w{};
  // sum of ceil(len / x) over the sequences is at most tokens / x + n_seqs
  w.max_fwd = s.tokens / (2 * s.TPT) + s.n_seqs;
  w.max_query = s.tokens / s.TPT + s.n_seqs;
  w.max_key = s.tokens / TILE + s.n_seqs;
  w.ld_stat = (s.tokens + 127) / 128 * 128;
  size_t off = 256;  // status word
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  w.counts = take(256);
  w.items = take((size_t)w.max_query * sizeof(Item));
  w.key_items = take((size_t)w.max_key * sizeof(Item));
  w.delta = take((size_t)s.heads * (size_t)w.ld_stat * sizeof(float));
  w.total = off;
  return w;
}

Source make_source(const Shape& s, const int32_t* starts, int tile, bool from_end, int group,
                   const Item* items, const int* count, int max_items, void* ws, int counter) {
  Source src{};
  if (s.n_seqs > SEARCH_SEQS) {
    src.items = items;
    src.count = count;
  }
  src.short_len = short_length(s.G);
  src.starts = starts;
  src.n_seqs = s.n_seqs;
  src.tile = tile;
  src.from_end = from_end;
  src.max_items = max_items;
  src.kv_heads = s.kv_heads;
  src.group = group;
  src.tokens = s.tokens;
  src.next = at<unsigned>(ws, COUNTERS) + 2 * counter;
  src.status = status_of(ws);
  return src;
}

int list_shift(long long max_cost) {
  int shift = 0;
  while ((max_cost >> shift) >= 1024) ++shift;
  return shift;
}

tsp_status launch_lists(const Shape& s, const int32_t* starts, const ListArgs& a, const ListArgs& b,
                        int* short_count, DevStatus* status, cudaStream_t stream) {
  packed_lists_kernel<<<b.tile ? 2 : 1, LIST_THREADS, 0, stream>>>(
      starts, s.n_seqs, s.tokens, a, b, short_length(s.G), short_count, status);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "packed attention: work list launch");
}

tsp_status make_query_map(CUtensorMap* map, const Shape& s, const void* base, int64_t ld) {
  const uint64_t dims[3] = {(uint64_t)s.d, (uint64_t)s.heads, (uint64_t)s.tokens};
  const uint64_t strides[2] = {(uint64_t)s.d * 2, (uint64_t)ld * 2};
  const uint32_t box[3] = {64, (uint32_t)s.G, (uint32_t)s.TPT};
  return make_tmap_3d_bf16(map, base, dims, strides, box);
}

int head_group(const Shape& s, long long l2_bytes) {
  // the heads split evenly over the fewest groups whose K and V fit
  const long long per_head = 4ll * std::max<long long>(s.tokens, 1) * s.d;
  const long long fit = std::max<long long>(1, l2_bytes / per_head);
  const long long groups = (s.kv_heads + fit - 1) / fit;
  return (int)((s.kv_heads + groups - 1) / groups);
}

tsp_status check_scale(const char* what, float scale) {
  if (!(scale > 0.f) || !std::isfinite(LOG2E * scale))
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": scale must be positive, and finite in base 2 as well");
  return TSP_OK;
}

tsp_status check_matrix(const char* what, const char* name, const void* p, int64_t ld, int64_t cols) {
  const std::string w = std::string(what) + ": " + name;
  if (!p) return fail(TSP_ERR_INVALID_ARG, w + " is a null pointer");
  if (!al16(p)) return fail(TSP_ERR_INVALID_ARG, w + " is not 16-byte aligned");
  if (ld < cols || ld % 8 || ld > (1ll << 32))
    return fail(TSP_ERR_INVALID_ARG, w + ": the row stride must be a multiple of 8 and hold the row");
  return TSP_OK;
}

}  // namespace packed
}  // namespace tsp

using namespace tsp;
using namespace tsp::packed;

extern "C" {

size_t tsp_packed_attention_workspace_bytes(int64_t tokens, int n_seqs, int heads, int kv_heads,
                                            int head_dim) {
  Shape s;
  if (make_shape("tsp_packed_attention_workspace_bytes", tokens, n_seqs, heads, kv_heads, head_dim,
                 &s) != TSP_OK)
    return 0;
  return make_workspace(s).total;
}

tsp_status tsp_packed_attention_fwd(int64_t tokens, int n_seqs, const int32_t* starts, int heads,
                                    int kv_heads, int head_dim, float scale, const tsp_bf16* q,
                                    int64_t ld_q, const tsp_bf16* k, int64_t ld_k, const tsp_bf16* v,
                                    int64_t ld_v, tsp_bf16* o, int64_t ld_o, float* lse,
                                    int64_t ld_lse, void* ws, void* stream) {
  TSP_GUARD_BEGIN
  const char* what = "tsp_packed_attention_fwd";
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
  if (lse && ((reinterpret_cast<uintptr_t>(lse) & 3u) || ld_lse < tokens))
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": lse misaligned, or its row stride below the tokens");
  if (o == q || o == k || o == v) return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": o aliases an input");
  TSP_TRY(check_ws(ws, what));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Workspace w = make_workspace(s);
  FwdParams p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.k = reinterpret_cast<const __nv_bfloat16*>(k);
  p.v = reinterpret_cast<const __nv_bfloat16*>(v);
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_v = ld_v;
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.ld_o = ld_o;
  p.lse = lse;
  p.ld_lse = ld_lse;
  // 72 MB of K and V in L2 at a time, as for the plan's attention
  p.src = make_source(s, starts, 2 * s.TPT, false, head_group(s, 72ll << 20), at<Item>(ws, w.items),
                      at<int>(ws, w.counts), (int)w.max_fwd, ws, 0);
  p.G = s.G;
  p.TPT = s.TPT;
  p.RU = s.RU;
  p.scale_log2 = LOG2E * scale;
  p.status = status_of(ws);
  p.limit_ns = wait_limit_ns();
  if (p.src.items != nullptr) {
    p.src.short_last = p.src.items + w.max_fwd - 1;
    p.src.short_count = at<int>(ws, w.counts) + 2;
    const ListArgs list{2 * s.TPT, 0, list_shift((tokens + TILE - 1) / TILE), at<Item>(ws, w.items),
                        at<int>(ws, w.counts), (int)w.max_fwd};
    TSP_TRY(launch_lists(s, starts, list, ListArgs{}, at<int>(ws, w.counts) + 2, p.status, st));
  }
  if (head_dim == 64) return launch_fwd<64>(s, p, q, ld_q, k, ld_k, v, ld_v, st);
  return launch_fwd<128>(s, p, q, ld_q, k, ld_k, v, ld_v, st);
  TSP_GUARD_END
}

}  // extern "C"
