// tile_walk.h - the order in which the persistent CTAs of a product take its tiles: `group` row tiles walk
// down one column tile, then the next column tile, then the next group (the last group may be shorter).
// Plain integers, for the host and the device.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TSP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TSP_HOST_DEVICE inline
#endif

namespace tsp {

// Row tiles of `tile_rows` rows that walk together, for A [m][k] and B [n][k] in bytes: about 32 MB of A where B does
// not fit the L2 well, else one. Never more than there are, so that group * (column tiles) is at most the number of
// tiles, which the caller keeps below 2^30.
inline int walk_group(int64_t m, int64_t n, int64_t k, int64_t tile_rows) {
  const int64_t g = n * k <= (48ll << 20) ? 1 : (32ll << 20) / (tile_rows * k);
  const int64_t tiles = (m + tile_rows - 1) / tile_rows;
  return (int)(g > tiles ? tiles : g < 1 ? 1 : g);
}

TSP_HOST_DEVICE void tile_coords(int tile, int num_p, int num_q, int group_p, int& tp, int& tq) {
  const int span = group_p * num_q;
  const int g = tile / span, r = tile - g * span;
  const int first = g * group_p;
  const int gm = group_p < num_p - first ? group_p : num_p - first;
  tp = first + r % gm;
  tq = r / gm;
}

}  // namespace tsp
