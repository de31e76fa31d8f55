// packed_short.cuh - sequences of a few tokens in the packed attention: whole warps instead of
// 128-row tiles.
//
// A sequence of at most 8 tokens, whose tokens times the heads of a group make at most 32 rows,
// would fill a fraction of its tiles and cost as much as they do. The element-wise warps of the
// tile kernels take those first, under the loads of their CTA's first item (behind the items it
// was a tail of 4 us or more, most of it the fetch of cold code), dealt out in a fixed order.
// Only the length and G decide, so a sequence's bits still do not depend on its neighbours.
//
// Forward, on the CUDA cores, P in fp32: a warp takes eight rows of a (sequence, key head); lane
// e holds columns [e d/32, (e + 1) d/32) of every row, K and V stay in registers, and four rows'
// scores with the eight keys are 32 sums over the warp, of which each lane ends with one. Bound
// by instructions (about 150 per row), below some hundred works by the latency of two loads.
//
// Backward, 16 rows x 8 keys as warp-wide products, P and dS rounded to bf16 as for tiles: dq in
// the query-side kernel by 16 rows, dk and dv in the key-side kernel by (sequence, key head).
// The forward's way took 806 instead of 383 us for 2000 sequences of 8 (32/8 of 128): a row has
// five products here, and their code outgrows the instruction caches. Both functions stay out of
// line, which keeps their registers out of the tile loops (in line the key side's cost 3% more).
//
// Against tiles alone, in us, forward | backward (query/key heads, width):
//                          8/2 of 64                32/8 of 128              16/16 of 64
//   one sequence of 8      5.8 / 6.4 | 13 / 17      6.4 / 7.0 | 18 / 19      6.0 / 6.4 | 12 / 17
//   100 of 8               6.6 / 11  | 20 / 27      15 / 29   | 32 / 70      10 / 45   | 23 / 108
//   2000 of 8              54 / 96   | 61 / 240     275 / 430 | 383 / 1044   131 / 721 | 206 / 1776
//   8 of 512, 20 of 6      12 / 12   | 50 / 49      33 / 36   | 136 / 137    19 / 25   | 71 / 86
//   64 of 100, 64 of 4     15 / 17   | 41 / 54      47 / 57   | 165 / 198    33 / 57   | 96 / 147
// Without a short sequence in the batch it costs 1 us of a backward.
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
  __device__ __forceinline__ int load(const Source& src) {
    if (src.items != nullptr) return min(__ldcg(src.short_count), src.n_seqs);
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
  __device__ __forceinline__ void get(const Source& src, int rank, int& start, int& len) const {
    if (src.items != nullptr) {
      const int2 it = __ldcg(reinterpret_cast<const int2*>(src.short_last - rank));  // an Item's
      start = it.x;
      len = it.y;
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
  if constexpr (E == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = u.x, v[1] = u.y;
  } else {
    v[0] = __ldg(p);
  }
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

// ------------------------------------------------------------------ backward
// Sixteen rows and the eight keys are one m16n8 product. With g = lane / 4 and c = lane % 4 a
// lane holds, of the scores, keys 2c and 2c + 1 of rows g and g + 8. Sums over d may run in any
// order, so a lane loads d/4 contiguous columns of its rows and keys; a product over rows or
// keys takes pairs of rows, whose two bf16 at one column a byte permutation puts side by side.
__device__ __forceinline__ void mma_k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {  // of an 8 x 8 matrix of 16 bits
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pair_of(uint32_t x, uint32_t y, int odd) {
  return __byte_perm(x, y, odd ? 0x7632 : 0x5410);
}

// N consecutive 32-bit words, 0 where there is no row.
template <int N>
__device__ __forceinline__ void load_words(const __nv_bfloat16* p, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint4 u = p != nullptr ? __ldg(reinterpret_cast<const uint4*>(p) + i / 4) : make_uint4(0u, 0u, 0u, 0u);
    w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
  }
}

// Where row r of a work lies: token r / G of the sequence, head r % G of the group.
struct RowAt {
  bool is;
  int token;
  long long row, head;
  __device__ __forceinline__ RowAt(int r, int G, int start, int len, int kv_head) {
    token = r / G;
    is = token < len;
    row = (long long)start + token;
    head = (long long)kv_head * G + (r - token * G);
  }
  __device__ __forceinline__ const __nv_bfloat16* in(const __nv_bfloat16* base, long long ld, int hd, int col) const {
    return is ? base + row * ld + head * hd + col : nullptr;
  }
};

// P and dS of rows [r0, r0 + 16), as bf16 pairs of keys 2c and 2c + 1 (rows g, g + 8), 0 where
// a row does not see a key. Delta is the sum of P dP.
template <int HD, class Params>
__device__ __forceinline__ void short_scores(const Params& p, int start, int len, int head, int r0,
                                             uint32_t (&pr)[2], uint32_t (&ds)[2]) {
  constexpr int N = HD / 8;  // words of a lane's d/4 columns
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, col = c * (HD / 4);
  const RowAt rows[2] = {RowAt(r0 + g, p.G, start, len, head), RowAt(r0 + g + 8, p.G, start, len, head)};
  float lse[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) lse[u] = rows[u].is ? __ldg(p.lse + rows[u].head * p.ld_lse + rows[u].row) : 0.f;
  auto product = [&](const __nv_bfloat16* a, long long ld_a, const __nv_bfloat16* b, long long ld_b, float (&d)[4]) {
    uint32_t a0[N], a1[N], bw[N];
    load_words<N>(rows[0].in(a, ld_a, HD, col), a0);
    load_words<N>(rows[1].in(a, ld_a, HD, col), a1);
    load_words<N>(g < len ? b + (long long)(start + g) * ld_b + head * HD + col : nullptr, bw);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; i += 2) mma_k16(d, a0[i], a1[i], a0[i + 1], a1[i + 1], bw[i], bw[i + 1]);
  };
  float s[4], dp[4];
  product(p.q, p.ld_q, p.k, p.ld_k, s);
  product(p.dout, p.ld_do, p.v, p.ld_v, dp);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float pe[2], part = 0.f;
    bool visible[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      visible[e] = rows[u].is && 2 * c + e <= rows[u].token;
      pe[e] = visible[e] ? ex2(fmaf(s[2 * u + e], p.scale_log2, -lse[u])) : 0.f;
      dp[2 * u + e] = visible[e] ? dp[2 * u + e] : 0.f;
      part = fmaf(pe[e], dp[2 * u + e], part);
    }
    part += __shfl_xor_sync(0xffffffffu, part, 1);
    part += __shfl_xor_sync(0xffffffffu, part, 2);
    pr[u] = pack_bf16x2(pe[0], pe[1]);
    ds[u] = pack_bf16x2(visible[0] ? pe[0] * (dp[2 * u] - part) : 0.f,
                        visible[1] ? pe[1] * (dp[2 * u + 1] - part) : 0.f);
  }
}

// Queries: a work is a (sequence, key head) and 16 of its rows; dq = scale dS K.
template <int HD, class Params>
__device__ __noinline__ void short_query_side(const Params& p, unsigned first, unsigned step) {
  if (p.src.short_len == 0) return;
  ShortFinder finder;
  const int n_short = finder.load(p.src);
  if (n_short <= 0) return;
  constexpr int W = HD / 8;  // a lane's columns of K, and of dq twice
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int parts = (p.src.short_len * p.G + 15) / 16;
  ShortWalk walk(first, step, (unsigned)(p.src.kv_heads * parts));
  for (; walk.rank < n_short; walk.next()) {
    int start, len;
    finder.get(p.src, (int)walk.rank, start, len);
    if (start < 0 || len > 8 || (long long)start + len > p.src.tokens) return;
    const int head = (int)walk.rem / parts, r0 = 16 * ((int)walk.rem - head * parts);
    if (r0 >= len * p.G) continue;
    uint32_t pr[2], ds[2];
    short_scores<HD>(p, start, len, head, r0, pr, ds);
    const RowAt rows[2] = {RowAt(r0 + g, p.G, start, len, head), RowAt(r0 + g + 8, p.G, start, len, head)};
#pragma unroll
    for (int half = 0; half < W / 8; ++half) {  // columns g W + 8 half + [0, 8) of K
      const __nv_bfloat16* k = p.k + (long long)(start + 2 * c) * p.ld_k + head * HD + g * W + 8 * half;
      uint32_t x[4], y[4];
      load_words<4>(2 * c < len ? k : nullptr, x);
      load_words<4>(2 * c + 1 < len ? k + p.ld_k : nullptr, y);
      float d[8][4];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] = 0.f;
        mma_k8(d[i], ds[0], ds[1], pair_of(x[i >> 1], y[i >> 1], i & 1));
      }
      // lane's results: rows g and g + 8, columns (2c + e) W + 8 half + i
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(d[2 * i][2 * u + e] * p.scale, d[2 * i + 1][2 * u + e] * p.scale);
          if (rows[u].is)
            *reinterpret_cast<uint4*>(p.dq + rows[u].row * p.ld_dq + rows[u].head * HD + (2 * c + e) * W + 8 * half) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
  }
}

// Keys: a work is a (sequence, key head), all its rows; dv = P^T dO, dk = scale dS^T Q. P and dS
// are formed again, as the two sides do for tiles.
template <int HD, class Params>
__device__ __noinline__ void short_key_side(const Params& p, unsigned first, unsigned step) {
  if (p.src.short_len == 0) return;
  ShortFinder finder;
  const int n_short = finder.load(p.src);
  if (n_short <= 0) return;
  constexpr int W = HD / 8;  // a lane's columns
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  ShortWalk walk(first, step, (unsigned)p.src.kv_heads);
  for (; walk.rank < n_short; walk.next()) {
    int start, len;
    finder.get(p.src, (int)walk.rank, start, len);
    if (start < 0 || len > 8 || (long long)start + len > p.src.tokens) return;
    const int head = (int)walk.rem;
    // [i][e]: columns g W + 2 i (e below 2) and g W + 2 i + 1 of key 2c + e % 2
    float dk[W / 2][4], dv[W / 2][4];
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) dk[i][e] = dv[i][e] = 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < len * p.G; r0 += 16) {
      uint32_t pr[2], ds[2];
      short_scores<HD>(p, start, len, head, r0, pr, ds);
      auto add = [&](const __nv_bfloat16* a, long long ld, const uint32_t (&b)[2], float (&d)[W / 2][4]) {
        const uint32_t b0 = transposed(b[0]), b1 = transposed(b[1]);
        uint32_t w[4][W / 2];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          load_words<W / 2>(RowAt(r0 + 2 * c + (u & 1) + 8 * (u >> 1), p.G, start, len, head).in(a, ld, HD, g * W),
                            w[u]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
          mma_k16(d[i], pair_of(w[0][i], w[1][i], 0), pair_of(w[0][i], w[1][i], 1), pair_of(w[2][i], w[3][i], 0),
                  pair_of(w[2][i], w[3][i], 1), b0, b1);
      };
      add(p.q, p.ld_q, ds, dk);
      add(p.dout, p.ld_do, pr, dv);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * c + e >= len) break;
      const long long row = start + 2 * c + e;
      auto store = [&](__nv_bfloat16* base, long long ld, const float (&d)[W / 2][4], float f) {
#pragma unroll
        for (int i = 0; i < W / 2; i += 4)
          *reinterpret_cast<uint4*>(base + row * ld + head * HD + g * W + 2 * i) =
              make_uint4(pack_bf16x2(d[i][e] * f, d[i][e + 2] * f), pack_bf16x2(d[i + 1][e] * f, d[i + 1][e + 2] * f),
                         pack_bf16x2(d[i + 2][e] * f, d[i + 2][e + 2] * f),
                         pack_bf16x2(d[i + 3][e] * f, d[i + 3][e + 2] * f));
      };
      store(p.dk, p.ld_dk, dk, p.scale);
      store(p.dv, p.ld_dv, dv, 1.f);
    }
    __syncwarp();
  }
}

}  // namespace packed
}  // namespace tsp
