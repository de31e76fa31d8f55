// packed_short.cuh - sequences of a few tokens in the packed attention's forward, on the CUDA
// cores.
//
// A sequence of at most 8 tokens, whose tokens times the heads of a group make at most 32 rows,
// would fill an eighth of its two 128-row tiles and cost as much as they do. Here a warp takes
// eight rows of such a (sequence, key head): lane e holds columns [e d/32, (e + 1) d/32) of
// every row, K and V stay in registers, and four rows' scores with the eight keys are 32 sums
// over the warp, of which each lane ends with one. Nothing is rounded but o. The softmax warps
// of the tile kernel do this before its items, under the first one's loads (behind the items it
// was a tail of 4 us or more, most of it the fetch of cold code), dealt out in a fixed order.
// Only the length and G decide, so a sequence's bits still do not depend on its neighbours.
//
// Bound by instructions (about 150 per row) and, below some hundred works, by the latency of
// two loads. Against tiles, in us:
//                          8/2 heads of 64   32/8 of 128   16/16 of 64   (query/key heads)
//   one sequence of 8          6.0 / 6.4       6.5 / 7.0      6.0 / 6.4
//   100 of 8                   6.6 / 10.9     15.6 / 29.5    10.1 / 45
//   2000 of 8                   54 / 96        272 / 430      130 / 721
//   8 of 512 and 20 of 6      12.1 / 11.9     32.6 / 35.6    18.6 / 25.0
#pragma once

#include "attention_math.cuh"
#include "packed_attention.cuh"

namespace tsp {
namespace packed {

// The short sequences, found by a whole warp: by rank among the starts in registers, or from
// the list.
struct ShortFinder {
  static constexpr int K = SEARCH_SEQS / 32;
  int st[K], ln[K];
  // Their number (0 where the starts are not in order).
  __device__ __forceinline__ int load(const ShortSource& src) {
    if (src.items != nullptr) return *src.short_count;
    bool bad = false;
    int n = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const int s = u * 32 + (threadIdx.x & 31);
      st[u] = ln[u] = 0;
      if (s < src.n_seqs) {
        const int a = src.starts[s], b = src.starts[s + 1];
        bad = bad || a < 0 || b < a || b > src.tokens;
        st[u] = a;
        ln[u] = b - a;
        n += ln[u] > 0 && ln[u] <= src.short_len;
      }
    }
    return __any_sync(0xffffffffu, bad) ? 0 : __reduce_add_sync(0xffffffffu, n);
  }
  // Sequence `rank` of the short ones (rank below their number).
  __device__ __forceinline__ void get(const ShortSource& src, int rank, int& start, int& len) const {
    if (src.items != nullptr) {
      const int2 s = src.short_items[rank];
      start = s.x;
      len = s.y;
      return;
    }
    const int lane = threadIdx.x & 31;
    start = len = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const unsigned mask = __ballot_sync(0xffffffffu, ln[u] > 0 && ln[u] <= src.short_len);
      const int here = __popc(mask);
      if (rank >= 0 && rank < here) {
        const bool mine = ((mask >> lane) & 1u) && __popc(mask & ((1u << lane) - 1u)) == rank;
        const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        start = __shfl_sync(0xffffffffu, st[u], from);
        len = __shfl_sync(0xffffffffu, ln[u], from);
      }
      rank -= here;
    }
  }
};

// This lane's E = d / 32 columns of a row.
template <int E>
__device__ __forceinline__ void row_part(const __nv_bfloat16* row, uint32_t (&v)[E / 2]) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + (threadIdx.x & 31) * (E / 2);
  // volatile: a loop's loads stay in the loop, where registers are short
  if constexpr (E == 4)
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v[0]) : "l"(p));
}
template <int E>
__device__ __forceinline__ void clear_part(uint32_t (&v)[E / 2]) {
#pragma unroll
  for (int e = 0; e < E / 2; ++e) v[e] = 0u;
}
template <int E>
__device__ __forceinline__ float part_value(const uint32_t (&v)[E / 2], int e) {
  return e & 1 ? bf16_hi(v[e / 2]) : bf16_lo(v[e / 2]);
}
// The rows of a sequence's keys or values, 0 behind it.
template <int HD>
__device__ __forceinline__ void load_rows(const __nv_bfloat16* base, long long ld, int len,
                                          uint32_t (&v)[8][HD / 64]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    clear_part<HD / 32>(v[j]);
    if (j < len) row_part<HD / 32>(base + j * ld, v[j]);
  }
}
template <int E>
__device__ __forceinline__ void store_part(__nv_bfloat16* row, const float (&v)[E], float f) {
  uint32_t* p = reinterpret_cast<uint32_t*>(row) + (threadIdx.x & 31) * (E / 2);
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f));
  else
    *p = pack_bf16x2(v[0] * f, v[1] * f);
}
template <int E>
__device__ __forceinline__ float dot_part(const uint32_t (&a)[E / 2], const uint32_t (&b)[E / 2]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    s = fmaf(bf16_lo(a[e]), bf16_lo(b[e]), s);
    s = fmaf(bf16_hi(a[e]), bf16_hi(b[e]), s);
  }
  return s;
}

// Sums of 32 values over the warp: lane l ends with that of value l.
__device__ __forceinline__ float sum_to_lanes(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 16; half > 0; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i)
      v[i] = (up ? v[half + i] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[half + i], half);
  }
  return v[0];
}
// Sum over the eight keys of the lane's row.
__device__ __forceinline__ float sum_keys(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

// Works (sequence, remainder below `per`), every `step`th from `first` on, without a division
// each.
struct ShortWalk {
  long long rank;
  unsigned rem, per, step_rank, step_rem;
  __device__ __forceinline__ ShortWalk(unsigned first, unsigned step, unsigned works_per_seq)
      : rank(first / works_per_seq), rem(first % works_per_seq), per(works_per_seq),
        step_rank(step / works_per_seq), step_rem(step % works_per_seq) {}
  __device__ __forceinline__ void next() {
    rank += step_rank;
    rem += step_rem;
    if (rem >= per) {
      rem -= per;
      ++rank;
    }
  }
};

// Partial products of four rows with eight keys, this lane's columns.
template <int E>
__device__ __forceinline__ void partial_products(const uint32_t (&a)[4][E / 2], const uint32_t (&b)[8][E / 2],
                                                 float (&s)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[8 * i + j] = dot_part<E>(a[i], b[j]);
}

// Forward. A work is a (sequence, key head) and 8 of its rows.
template <int HD, class Params>
__device__ __forceinline__ void short_forward(const Params& p, unsigned first, unsigned step) {
  constexpr int E = HD / 32;
  if (p.src.short_len == 0) return;
  prior_kernel_done();  // the list
  ShortFinder finder;
  const int n_short = finder.load(p.src);
  if (n_short <= 0) return;
  const int lane = threadIdx.x & 31;
  const int parts = (p.src.short_len * p.G + 7) / 8;
  ShortWalk walk(first, step, (unsigned)(p.src.kv_heads * parts));
  for (; walk.rank < n_short; walk.next()) {
    int start, len;
    finder.get(p.src, (int)walk.rank, start, len);
    if (start < 0 || len > 8 || (long long)start + len > p.src.tokens) return;
    const int head = (int)walk.rem / parts, part = (int)walk.rem - head * parts;
    if (8 * part >= len * p.G) continue;
    uint32_t k[8][E / 2], v[8][E / 2];
    load_rows<HD>(p.k + (long long)start * p.ld_k + head * HD, p.ld_k, len, k);
    load_rows<HD>(p.v + (long long)start * p.ld_v + head * HD, p.ld_v, len, v);
    // rolled loops: the code is cold in most calls, and its fetch costs more than it computes
#pragma unroll 1
    for (int r0 = 8 * part; r0 < min(8 * part + 8, len * p.G); r0 += 4) {
      uint32_t q[4][E / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ti = (r0 + i) / p.G;
        const long long qh = (long long)head * p.G + (r0 + i - ti * p.G);
        clear_part<E>(q[i]);
        if (ti < len) row_part<E>(p.q + (long long)(start + ti) * p.ld_q + qh * HD, q[i]);
      }
      float s[32];
      partial_products<E>(q, k, s);
      const int r = r0 + (lane >> 3), t = r / p.G;
      const float sum = sum_to_lanes(s);
      const bool visible = (lane & 7) <= t;
      const float x = visible ? sum * p.scale_log2 : -INFINITY;
      float m = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
      const float pr = visible ? ex2(x - m) : 0.f;
      const float l = sum_keys(pr);
      if (p.lse != nullptr && (lane & 7) == 0 && t < len)
        p.lse[((long long)head * p.G + (r - t * p.G)) * p.ld_lse + start + t] = m + log2f(l);
      const float inv = 1.f / l;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int ti = __shfl_sync(0xffffffffu, t, 8 * i);
        if (ti >= len) break;
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float pj = __shfl_sync(0xffffffffu, pr, 8 * i + j);
          if (j <= ti) {  // 0 times a value that is not finite is not 0
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(pj, part_value<E>(v[j], e), o[e]);
          }
        }
        const long long qh = (long long)head * p.G + (r0 + i - ti * p.G);
        store_part<E>(p.o + (long long)(start + ti) * p.ld_o + qh * HD, o, __shfl_sync(0xffffffffu, inv, 8 * i));
      }
    }
  }
}

}  // namespace packed
}  // namespace tsp
