// packed_attention.cuh - shapes, work lists and workspace shared by the forward and the
// backward of the packed (variable-length, grouped-head) attention.
#pragma once

#include "tsp_device.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace packed {

constexpr int TILE = 128;                  // rows of a tensor-core tile, and keys per key tile
constexpr uint32_t BOX_BYTES = 128 * 128;  // 128 rows x 64 bf16 in shared memory
constexpr float LOG2E = 1.4426950408889634f;
constexpr size_t COUNTERS = 128;           // byte offset in the workspace's first 256 bytes

// One CTA's share of a sequence: the tile (or pair of tiles) that begins at token q0.
struct Item {
  int start;  // the sequence's first row
  int len;    // and its tokens
  int q0;
  int head;  // key head (set by find_item)
};

struct Shape {
  long long tokens;  // rows of q, k, v and o
  int n_seqs;
  int heads, kv_heads, d;
  int G;    // query heads per key head
  int TPT;  // tokens per 128-row query tile: row = token * G + head of the group
  int RU;   // rows in use, TPT * G <= 128
};

// Sequences of up to this many tokens are short: at most 8, and 32 rows of tokens x heads of a
// group (packed_short.cuh takes them, tiles the others).
inline int short_length(int G) { return 32 / G < 8 ? 32 / G : 8; }

// Workspace (byte offsets from its 256-byte aligned start).
struct Workspace {
  // the first 256 bytes: the status word, and from COUNTERS on two words per kernel for Walk
  size_t counts;  // int[3]: items in each list
  size_t items;   // forward, or query side of the backward
  size_t key_items;
  size_t delta;   // [heads][ld_stat] fp32
  size_t total;
  long long max_fwd, max_query, max_key;  // capacity of the lists
  long long ld_stat;
};

// A list of items: one per `tile` tokens of every sequence, the costliest first. The cost
// is the number of 128-key tiles up to the item's last token (streamed == 0), or the number
// of `streamed`-token query tiles from its first key on.
struct ListArgs {
  int tile;
  int streamed;
  int shift;  // cost >> shift < 1024
  Item* items;
  int* count;
  int max_items;
};

// Where a kernel takes its items from: a list made by launch_lists, or, for up to
// SEARCH_SEQS sequences, the starts themselves (items == nullptr).
constexpr int SEARCH_SEQS = 128;
struct Source {
  const Item* items;
  const int* count;
  const int32_t* starts;
  int n_seqs;
  int tile;      // tokens per item
  int from_end;  // the costliest items are the first ones of a sequence (key side)
  int max_items;
  int kv_heads;
  int group;     // key heads whose CTAs interleave
  long long tokens;
  unsigned* next;  // [2] in the workspace: works handed out beyond the first of each CTA, and
                   // CTAs that are done; both 0 before and after a launch
  DevStatus* status;
  int short_len;            // sequences of up to so many tokens are no items
  const Item* short_last;   // with a list: those sequences, backwards from here
  const int* short_count;
};

#ifdef __CUDACC__
// Work w of a launch as an item and its key head, by a whole warp; false if there are no more
// than w works, or if the starts are not in order. The works of a group of key heads come
// item by item, the costliest first, every head of the group at each item.
//
// Up to SEARCH_SEQS sequences the item comes from the starts themselves: items of equal
// distance b from the cheap end of their sequence cost the same, and sum max(0, nb - b) items
// lie at b or further, so b comes from a binary search over warp sums and the sequence from a
// rank among those with more than b items. About a microsecond, which the persistent kernels
// spend beside their products, against 5 for a kernel that writes the list.
static __device__ __forceinline__ bool find_item(const Source& src, unsigned w, Item& it) {
  constexpr int K = SEARCH_SEQS / 32;
  const int lane = threadIdx.x & 31;
  int nb[K], st[K], ln[K];
  int total;
  if (src.items == nullptr) {
    bool bad = false;
    total = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const int s = u * 32 + lane;
      st[u] = ln[u] = nb[u] = 0;
      if (s < src.n_seqs) {
        const int a = src.starts[s], b = src.starts[s + 1];
        bad = bad || a < 0 || b < a || b > src.tokens;
        st[u] = a;
        ln[u] = b - a;
        nb[u] = ln[u] <= src.short_len ? 0 : (int)(((long long)ln[u] + src.tile - 1) / src.tile);
      }
      total += nb[u];
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (threadIdx.x == 0) record_error(src.status, kStatusInvalid, SITE_PACKED_STARTS);
      return false;
    }
    total = __reduce_add_sync(0xffffffffu, total);
  } else {
    // past L1: the key side reads the list without having waited for the kernel that wrote it
    // (the query side has, before it let the key side start)
    total = min(__ldcg(src.count), src.max_items);
  }
  if (total <= 0 || w >= (unsigned long long)total * (unsigned)src.kv_heads) return false;
  const unsigned per_group = (unsigned)total * (unsigned)src.group;
  const int grp = (int)(w / per_group);
  const int in_g = min(src.group, src.kv_heads - grp * src.group);
  const int rem = (int)(w - grp * per_group);
  const int idx = rem / in_g;
  it.head = grp * src.group + (rem - idx * in_g);
  if (src.items != nullptr) {
    const int4 listed = __ldcg(reinterpret_cast<const int4*>(src.items + idx));  // an Item
    it.start = listed.x;
    it.len = listed.y;
    it.q0 = listed.z;
  } else {
    auto from = [&](int b) {
      int c = 0;
#pragma unroll
      for (int u = 0; u < K; ++u) c += max(0, nb[u] - b);
      return __reduce_add_sync(0xffffffffu, c);
    };
    int most = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) most = max(most, nb[u]);
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, most) - 1;  // the largest b with from(b) > idx
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (from(mid) > idx) lo = mid;
      else hi = mid - 1;
    }
    int r = idx - from(lo + 1);
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const unsigned mask = __ballot_sync(0xffffffffu, nb[u] > lo);
      const int here = __popc(mask);
      if (r >= 0 && r < here) {
        const bool mine = ((mask >> lane) & 1u) && __popc(mask & ((1u << lane) - 1u)) == r;
        const int from_lane = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        it.start = __shfl_sync(0xffffffffu, st[u], from_lane);
        it.len = __shfl_sync(0xffffffffu, ln[u], from_lane);
        const int n = __shfl_sync(0xffffffffu, nb[u], from_lane);
        it.q0 = (src.from_end ? n - 1 - lo : lo) * src.tile;
      }
      r -= here;
    }
  }
  // the list may only be trusted as far as this call's own buffers
  return it.start >= 0 && it.q0 >= 0 && it.len > it.q0 &&
         (long long)it.start + it.len <= src.tokens;
}

// The items of a persistent CTA, one after the other, by a whole warp. The first work is the
// CTA's own number; the others are drawn from a counter, so the CTAs that finish early take
// what is left. The list falls in cost, hence what is left last is short.
struct Walk {
  bool begun = false;
  // Moves on to the next item (the first call: to the first); head -1 at the end.
  __device__ __forceinline__ void next(const Source& src, Item& it) {
    unsigned w = blockIdx.x;
    if (begun) {
      if ((threadIdx.x & 31) == 0) w = gridDim.x + atomicAdd(src.next, 1u);
      w = __shfl_sync(0xffffffffu, w, 0);
    }
    begun = true;
    if (!find_item(src, w, it)) it.head = -1;
  }
  // Once per CTA, after its last next(), by one thread: the last CTA leaves the counters at 0.
  __device__ __forceinline__ void end(const Source& src) {
    __threadfence();
    if (atomicAdd(src.next + 1, 1u) == gridDim.x - 1u) {
      src.next[0] = 0u;
      src.next[1] = 0u;
    }
  }
};

// The start of a persistent CTA: warp 0 has set up the barriers and goes on to its first
// loads, the others meet (tensor memory allocated, shared memory cleared) and see what warp 0
// wrote before.
template <int THREADS>
static __device__ __forceinline__ void start_arrive() {
  asm volatile("barrier.cta.arrive 1, %0;" ::"n"(THREADS) : "memory");
}
template <int THREADS>
static __device__ __forceinline__ void start_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Stores one accumulator row per lane (32 columns as 16 packed bf16 pairs), 16 bytes at a
// time. Lane by lane that would touch 32 lines per instruction; a 4 x 4 exchange of 16-byte
// chunks inside groups of four lanes first lets four lanes write 64 contiguous bytes of one
// row. `dst[k]` is the first of the 32 columns of row k of the lane's group of four, or
// nullptr where that row is not written.
static __device__ __forceinline__ void store_rows(uint32_t (&v)[16], __nv_bfloat16* const (&dst)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int bit = 0; bit < 2; ++bit) {
    const bool up = (lane >> bit) & 1;
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      // chunks (0,1), (2,3) with the neighbour; then (0,2), (1,3) with the next but one
      const int lo = bit == 0 ? 2 * pair : pair, hi = lo + (1 << bit);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t give = up ? v[4 * lo + e] : v[4 * hi + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1 << bit);
        if (up) v[4 * lo + e] = got;
        else v[4 * hi + e] = got;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (dst[k] != nullptr)
      reinterpret_cast<uint4*>(dst[k])[lane & 3] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
}

// The row pointers of the lane's group of four, from each lane's own (nullptr: not written).
static __device__ __forceinline__ void group_rows(__nv_bfloat16* mine, __nv_bfloat16* (&dst)[4]) {
  const unsigned long long m = reinterpret_cast<unsigned long long>(mine);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    dst[k] = reinterpret_cast<__nv_bfloat16*>(__shfl_sync(0xffffffffu, m, ((threadIdx.x & 31) & ~3) + k));
}
#endif

tsp_status make_shape(const char* what, int64_t tokens, int n_seqs, int heads, int kv_heads,
                      int head_dim, Shape* s);
Workspace make_workspace(const Shape& s);
// Fills one or two lists (b.tile == 0: one) from the sequence starts, on the device.
tsp_status launch_lists(const Shape& s, const int32_t* starts, const ListArgs& a, const ListArgs& b,
                        int* short_count, DevStatus* status, cudaStream_t stream);
Source make_source(const Shape& s, const int32_t* starts, int tile, bool from_end, int group,
                   const Item* items, const int* count, int max_items, void* ws, int counter);
int list_shift(long long max_cost);
// Query heads grouped by key head: box of 64 columns x G heads x TPT tokens.
tsp_status make_query_map(CUtensorMap* map, const Shape& s, const void* base, int64_t ld);
// Key heads whose K and V share L2 (CTAs of a group run together).
int head_group(const Shape& s, long long l2_bytes);
// The kernels multiply the scores by scale log2(e): it may not overflow, or a score of 0 is NaN.
tsp_status check_scale(const char* what, float scale);
tsp_status check_matrix(const char* what, const char* name, const void* p, int64_t ld, int64_t cols);

}  // namespace packed
}  // namespace tsp
