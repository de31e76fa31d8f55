// packed_attention.cuh - shapes, work lists and workspace shared by the forward and the
// backward of the packed (variable-length, grouped-head) attention.
#pragma once

#include "tsp_device.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace packed {

constexpr int TILE = 128;                  // rows of a tensor-core tile, and keys per key tile
constexpr uint32_t BOX_BYTES = 128 * 128;  // 128 rows x 64 bf16 in shared memory

// One CTA's share of a sequence: the tile (or pair of tiles) that begins at token q0.
struct Item {
  int start;  // the sequence's first row
  int len;    // and its tokens
  int q0;
  int unused;
};

struct Shape {
  long long tokens;  // rows of q, k, v and o
  int n_seqs;
  int heads, kv_heads, d;
  int G;    // query heads per key head
  int TPT;  // tokens per 128-row query tile: row = token * G + head of the group
  int RU;   // rows in use, TPT * G <= 128
};

// Workspace (byte offsets from its 256-byte aligned start).
struct Workspace {
  size_t counts;  // int[2]: items in each list
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

tsp_status make_shape(const char* what, int64_t tokens, int n_seqs, int heads, int kv_heads,
                      int head_dim, Shape* s);
Workspace make_workspace(const Shape& s);
// Fills one or two lists (b.tile == 0: one) from the sequence starts, on the device.
tsp_status launch_lists(const Shape& s, const int32_t* starts, const ListArgs& a, const ListArgs& b,
                        DevStatus* status, cudaStream_t stream);
int list_shift(long long max_cost);
// Query heads grouped by key head: box of 64 columns x G heads x TPT tokens.
tsp_status make_query_map(CUtensorMap* map, const Shape& s, const void* base, int64_t ld);
// Key heads whose K and V share L2 (CTAs of a group run together).
int head_group(const Shape& s, long long l2_bytes);
tsp_status check_matrix(const char* what, const char* name, const void* p, int64_t ld, int64_t cols);

}  // namespace packed
}  // namespace tsp
