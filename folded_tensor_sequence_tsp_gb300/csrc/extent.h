// extent.h - where a matrix lies in memory, and whether two of them share a byte. Plain integers on the host.
#pragma once

#include <cstdint>

namespace tsp {

// `rows` rows of `width` bytes, `stride` >= width bytes apart.
struct Extent {
  uint64_t at, rows, width, stride;
};

inline Extent extent(const void* p, int64_t rows, int64_t width, int64_t stride) {
  Extent e{reinterpret_cast<uintptr_t>(p), (uint64_t)rows, (uint64_t)width, (uint64_t)stride};
  if (e.rows == 0 || e.width == 0) e.rows = e.width = 0;
  else if (e.rows == 1 || e.stride == e.width) e.width *= e.rows, e.rows = 1, e.stride = e.width;  // one run
  return e;
}

// The byte behind the last one (the largest number where that does not fit).
inline uint64_t extent_end(const Extent& e) {
  const uint64_t most = ~0ull - e.at - e.width;
  return e.rows - 1 > most / e.stride ? ~0ull : e.at + (e.rows - 1) * e.stride + e.width;
}

// One run beside rows: does the first row that ends behind the run's start begin before its end?
inline bool run_overlaps(const Extent& run, const Extent& rows) {
  const uint64_t end = rows.at + rows.width;
  const uint64_t j = run.at < end ? 0 : (run.at - end) / rows.stride + 1;
  return j < rows.rows && rows.at + j * rows.stride < run.at + run.width;
}

// Rows that interleave without a common byte are told from others where both matrices have the same stride, or one is
// a single run; with unlike strides, one that begins before the other's end counts as an overlap.
inline bool overlaps(const Extent& a, const Extent& b) {
  if (a.rows == 0 || b.rows == 0) return false;
  if (a.at >= extent_end(b) || b.at >= extent_end(a)) return false;
  if (a.rows == 1) return run_overlaps(a, b);
  if (b.rows == 1) return run_overlaps(b, a);
  if (a.stride != b.stride) return true;
  // row i of a and row i + d of b are e + (d - d0) stride bytes apart, 0 <= e < stride: only d0 and the one before can meet
  const int64_t s = (int64_t)a.stride, apart = (int64_t)(b.at - a.at);
  const int64_t e = (apart % s + s) % s, d0 = (e - apart) / s;
  auto both_have = [&](int64_t d) { return d > -(int64_t)a.rows && d < (int64_t)b.rows; };
  return (e < (int64_t)a.width && both_have(d0)) || (s - e < (int64_t)b.width && both_have(d0 - 1));
}

}  // namespace tsp
