// quantize.cu - e4m3 values with an fp32 scale for each block of 128, from bf16 or fp32:
//     scale = max|x| / 448 over the block (1 for zeros, at least 2^-126), q = e4m3(x / scale)
// in the forms that the products of a linear layer read (matmul_e4m3.cu):
//   rows       y  [rows][width]: a scale for 128 columns of one row
//   columns    yt [width][rows]: the transpose, a scale for 128 rows of one column
//   tiles      one scale for 128 x 128 values: y and its transpose hold the same values
//
// Bound: HBM for rows and tiles (16384 x 4096 bf16 rows: 31 us, 0.95 of the copy rate; 11008 x 4096 fp32 tiles in
// both layouts: 43 us, 0.92), the arithmetic of two quotients a value for both layouts with scales of their own
// (16384 x 4096 bf16: 54 us, 0.74). x is read once, whatever is written. In rows eight lanes hold a block, 16
// values each, so that a divisor is worked out for 16 values (with four per lane: 104 us). What needs a
// column's largest value or a transpose takes a tile of 128 x 128 per CTA: each warp holds 16 rows as they are
// stored, the rows' and columns' maxima meet in shared memory, where one thread each makes the divisors (in
// every lane: 135 us for 16384 x 4096), and the transposed bytes go through a 16 KB tile there (16-byte chunks,
// swizzled by their column) so that both layouts are written in runs of 128 bytes. With quotients of six
// operations for two values in place of QuickQuotient's two: 34, 51 and 67 us. Rows of odd width or off their boundary
// are read and written a value at a time (16384 x 4095 bf16: rows 80 us, both layouts 108; 11008 x 4095 fp32 tiles: 50).
#include <type_traits>

#include "e4m3.cuh"
#include "extent.h"
#include "tsp_internal.h"

namespace tsp {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 128;  // values under one scale, and the side of a tile

struct QuantParams {
  long long rows, width;
  const void* x;
  long long ld_x;
  uint8_t* y;
  long long ld_y;
  float* scales;
  uint8_t* yt;
  long long ld_yt;
  float* scales_t;
};

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(fabsf(v)); }

template <class Q>
__device__ __forceinline__ uint32_t quantize4(const Q& by, const float (&v)[4]) {
  float a = v[0], b = v[1], c = v[2], d = v[3];
  by.pair(a, b);
  by.pair(c, d);
  return to_e4m3x4(a, b, c, d);
}

template <bool VEC>
__device__ __forceinline__ void store4(uint8_t* y, int left, uint32_t q) {
  if constexpr (VEC) {
    if (left > 0) *reinterpret_cast<uint32_t*>(y) = q;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) y[e] = (uint8_t)(q >> (8 * e));
  }
}

// Rows that start on 16 bytes: eight lanes per block of 128 columns, 16 values each (two runs of 8 in bf16,
// four of 4 in fp32), so that a scale and its reciprocal are worked out for 16 values at once. A warp takes
// eight blocks.
template <bool F32>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantParams p) {
  constexpr int U = 2, PER = F32 ? 4 : 8, RUNS = 16 / PER;
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const uint32_t groups = (uint32_t)((p.width + kBlock - 1) / kBlock);
  const uint32_t blocks = (uint32_t)p.rows * groups;  // below 2^31: checked by the caller
  const uint32_t first = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (4 * U) + (lane >> 3);
  dependents_may_start();
  prior_kernel_done();
  uint4 raw[U][RUNS];
  uint32_t row[U];
  int col[U];  // of the block
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t b = first + 4 * u;
    row[u] = b / groups;
    col[u] = (int)(b - row[u] * groups) * kBlock;
    const int es = F32 ? 4 : 2;
    const uint8_t* from = static_cast<const uint8_t*>(p.x) + ((long long)row[u] * p.ld_x + col[u]) * es;
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int c = PER * (8 * k + sub);
      raw[u][k] = make_uint4(0u, 0u, 0u, 0u);
      if (b < blocks && col[u] + c < p.width) raw[u][k] = __ldcs(reinterpret_cast<const uint4*>(from + c * es));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t b = first + 4 * u;
    uint32_t top = 0u;
    float v[16];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const uint32_t w[4] = {raw[u][k].x, raw[u][k].y, raw[u][k].z, raw[u][k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F32) {
          v[4 * k + e] = __uint_as_float(w[e]);
          top = max(top, w[e] & 0x7fffffffu);
        } else {
          v[8 * k + 2 * e] = bf16_lo(w[e]);
          v[8 * k + 2 * e + 1] = bf16_hi(w[e]);
          top = __vmaxu2(top, w[e] & 0x7fff7fffu);  // the two halves apart
        }
      }
    }
    if constexpr (!F32) top = max(top << 16, top & 0xffff0000u);
#pragma unroll
    for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = e4m3_scale(top);
    const QuickQuotient quick(scale);
    if (sub == 0 && b < blocks) p.scales[b] = scale;
    uint8_t* to = p.y + (long long)row[u] * p.ld_y + col[u];
    auto write = [&](const auto& by) {
#pragma unroll
      for (int k = 0; k < RUNS; ++k) {
        const int c = PER * (8 * k + sub);
        if (b >= blocks || col[u] + c >= p.width) continue;
        const float four[4] = {v[PER * k], v[PER * k + 1], v[PER * k + 2], v[PER * k + 3]};
        const uint32_t lo = quantize4(by, four);
        if constexpr (F32) {
          *reinterpret_cast<uint32_t*>(to + c) = lo;
        } else {
          const float more[4] = {v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]};
          *reinterpret_cast<uint2*>(to + c) = make_uint2(lo, quantize4(by, more));
        }
      }
    };
    if (__all_sync(0xffffffffu, quick.ok)) write(quick);
    else write(Quotient(scale));
  }
}

// Other rows: one warp per row and 128 columns, four single values per lane.
template <bool F32>
__global__ void __launch_bounds__(kThreads) quantize_any_rows_kernel(const QuantParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t groups = (uint32_t)((p.width + kBlock - 1) / kBlock);
  const uint32_t blocks = (uint32_t)p.rows * groups;
  const uint32_t b = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  dependents_may_start();
  prior_kernel_done();
  if (b >= blocks) return;
  const uint32_t row = b / groups;
  const int col = (int)(b - row * groups) * kBlock + lane;
  float v[4];
  uint32_t top = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = 0.f;
    if (col + 32 * e < p.width) {
      const long long at = (long long)row * p.ld_x + col + 32 * e;
      v[e] = F32 ? static_cast<const float*>(p.x)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.x)[at]);
    }
    top = max(top, magnitude(v[e]));
  }
  const float scale = e4m3_scale(__reduce_max_sync(0xffffffffu, top));
  if (lane == 0) p.scales[b] = scale;
  const uint32_t q = quantize4(Quotient(scale), v);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + 32 * e < p.width) p.y[(long long)row * p.ld_y + col + 32 * e] = (uint8_t)(q >> (8 * e));
}

// The scale of a row or column of a tile and the constants of a quick quotient by it, worked out once; lo is
// negative where that quotient will not do.
struct __align__(16) Divisor {
  float hi, lo, scale;
};
__device__ __forceinline__ Divisor divisor(uint32_t top) {
  const float scale = e4m3_scale(top);
  const QuickQuotient quick(scale);
  return {quick.hi, quick.ok ? quick.lo : -1.f, scale};
}
// The quotient by it, of either kind.
template <bool QUICK>
__device__ __forceinline__ auto quotient(const Divisor& d) {
  if constexpr (QUICK) {
    QuickQuotient by(1.f);
    by.hi = d.hi, by.lo = d.lo;
    return by;
  } else {
    return Quotient(d.scale);
  }
}
// One branch for all of a warp's divisors: f(std::true_type) where a quick quotient does for each lane's.
template <class F>
__device__ __forceinline__ void with_quotients(bool ok, F f) {
  if (__all_sync(0xffffffffu, ok)) f(std::true_type());
  else f(std::false_type());
}

// One CTA per tile of 128 x 128. TILE: one scale for all of it. VEC: the width is a multiple of 4 and every
// row starts on 16 (fp32) or 8 (bf16) bytes, in y on 4. A warp holds 16 rows, a lane four columns of
// them as they are stored; the rows' and columns' largest values meet in shared memory, where one
// thread each makes the divisors. CTAs per SM as measured: bf16 2, 3 and 4: 69, 61 and 54 us for 16384 x 4096; fp32
// with a scale per row and column 2 and 3: 80 and 108 us. vec_t: yt's rows start on 16 bytes.
template <bool F32, bool TILE, bool VEC>
__global__ void __launch_bounds__(kThreads, F32 ? (TILE ? 3 : 2) : 4) quantize_tile_kernel(const QuantParams p, int vec_t) {
  __shared__ __align__(16) uint8_t turned[kBlock * kBlock];
  __shared__ __align__(16) uint32_t col_tops[kThreads / 32][kBlock];
  __shared__ uint32_t row_tops[kBlock];
  __shared__ Divisor row_div[kBlock], col_div[kBlock];
  constexpr int WORDS = F32 ? 4 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tiles_w = (uint32_t)((p.width + kBlock - 1) / kBlock), tiles_r = (uint32_t)((p.rows + kBlock - 1) / kBlock);
  const uint32_t tr = blockIdx.x / tiles_w, tc = blockIdx.x - tr * tiles_w;
  const long long row0 = (long long)tr * kBlock + 16 * warp, col = (long long)tc * kBlock + 4 * lane;
  const int left = (int)min(p.width - col, 4ll), rows_left = (int)min(p.rows - row0, 16ll);
  dependents_may_start();
  prior_kernel_done();
  uint32_t raw[16][WORDS];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
#pragma unroll
    for (int e = 0; e < WORDS; ++e) raw[r][e] = 0u;
    if (r >= rows_left || left <= 0) continue;
    const long long at = (row0 + r) * p.ld_x + col;
    if constexpr (VEC && F32) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(p.x) + at));
      raw[r][0] = u.x, raw[r][1] = u.y, raw[r][2] = u.z, raw[r][3] = u.w;
    } else if constexpr (VEC) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.x) + at));
      raw[r][0] = u.x, raw[r][1] = u.y;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) {
          if constexpr (F32) raw[r][e] = static_cast<const uint32_t*>(p.x)[at + e];
          else raw[r][e >> 1] |= (uint32_t)static_cast<const uint16_t*>(p.x)[at + e] << (16 * (e & 1));
        }
    }
  }
  auto four = [&](int r, float (&v)[4]) {
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(raw[r][e]);
    } else {
      v[0] = bf16_lo(raw[r][0]), v[1] = bf16_hi(raw[r][0]), v[2] = bf16_lo(raw[r][1]), v[3] = bf16_hi(raw[r][1]);
    }
  };
  auto one = [&](int r, int e) {
    if constexpr (F32) return __uint_as_float(raw[r][e]);
    else return (e & 1) ? bf16_hi(raw[r][e >> 1]) : bf16_lo(raw[r][e >> 1]);
  };

  // largest magnitudes, as bits: of each row (not for TILE), and of this lane's columns
  uint32_t tops[WORDS];
#pragma unroll
  for (int e = 0; e < WORDS; ++e) tops[e] = 0u;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    uint32_t of_row = 0u;
#pragma unroll
    for (int e = 0; e < WORDS; ++e) {
      const uint32_t m = raw[r][e] & (F32 ? 0x7fffffffu : 0x7fff7fffu);
      tops[e] = F32 ? max(tops[e], m) : __vmaxu2(tops[e], m);
      of_row = F32 ? max(of_row, m) : __vmaxu2(of_row, m);
    }
    if constexpr (!TILE) {
      if constexpr (!F32) of_row = max(of_row << 16, of_row & 0xffff0000u);
      of_row = __reduce_max_sync(0xffffffffu, of_row);
      if (lane == r) row_tops[16 * warp + r] = of_row;
    }
  }
  uint32_t top[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    top[e] = F32 ? tops[F32 ? e : 0] : (e & 1) ? tops[e >> 1] & 0xffff0000u : tops[e >> 1] << 16;
  if constexpr (TILE) {
    const uint32_t t = __reduce_max_sync(0xffffffffu, max(max(top[0], top[1]), max(top[2], top[3])));
    if (lane == 0) row_tops[warp] = t;
  } else {
    *reinterpret_cast<uint4*>(&col_tops[warp][4 * lane]) = make_uint4(top[0], top[1], top[2], top[3]);
  }
  __syncthreads();
  if constexpr (TILE) {
    const Divisor by = divisor(__reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? row_tops[lane] : 0u));
    if (threadIdx.x == 0) {
      if (p.y) p.scales[(long long)tr * tiles_w + tc] = by.scale;
      if (p.yt) p.scales_t[(long long)tc * tiles_r + tr] = by.scale;
    }
    uint32_t q[16];
    with_quotients(by.lo >= 0.f, [&](auto quick) {
      const auto divide = quotient<quick.value>(by);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float v[4];
        four(r, v);
        q[r] = quantize4(divide, v);
        if (p.y && r < rows_left) store4<VEC>(p.y + (row0 + r) * p.ld_y + col, left, q[r]);
      }
    });
    if (!p.yt) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // byte e of four rows
        const uint32_t lo = __byte_perm(q[4 * k], q[4 * k + 1], e | ((4 + e) << 4));
        const uint32_t hi = __byte_perm(q[4 * k + 2], q[4 * k + 3], e | ((4 + e) << 4));
        w[k] = __byte_perm(lo, hi, 0x5410);
      }
      *reinterpret_cast<uint4*>(turned + (4 * lane + e) * kBlock + ((warp ^ (lane & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    const int i = threadIdx.x & (kBlock - 1);
    if (threadIdx.x < kBlock) {
      const Divisor d = divisor(row_tops[i]);
      row_div[i] = d;
      if (p.y && (long long)tr * kBlock + i < p.rows) p.scales[((long long)tr * kBlock + i) * tiles_w + tc] = d.scale;
    } else {
      uint32_t t = col_tops[0][i];
#pragma unroll
      for (int k = 1; k < kThreads / 32; ++k) t = max(t, col_tops[k][i]);
      const Divisor d = divisor(t);
      col_div[i] = d;
      if ((long long)tc * kBlock + i < p.width) p.scales_t[((long long)tc * kBlock + i) * tiles_r + tr] = d.scale;
    }
    __syncthreads();
    if (p.y) {
      with_quotients(row_div[16 * warp + (lane & 15)].lo >= 0.f, [&](auto quick) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (r >= rows_left) break;
          float v[4];
          four(r, v);
          store4<VEC>(p.y + (row0 + r) * p.ld_y + col, left, quantize4(quotient<quick.value>(row_div[16 * warp + r]), v));
        }
      });
    }
    const Divisor by[4] = {col_div[4 * lane], col_div[4 * lane + 1], col_div[4 * lane + 2], col_div[4 * lane + 3]};
    with_quotients(min(min(by[0].lo, by[1].lo), min(by[2].lo, by[3].lo)) >= 0.f, [&](auto quick) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const auto divide = quotient<quick.value>(by[e]);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float v[4] = {one(4 * k, e), one(4 * k + 1, e), one(4 * k + 2, e), one(4 * k + 3, e)};
          w[k] = quantize4(divide, v);
        }
        *reinterpret_cast<uint4*>(turned + (4 * lane + e) * kBlock + ((warp ^ (lane & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    });
  }
  __syncthreads();
  // 16 rows of x of one column per thread and step
#pragma unroll
  for (int i = 0; i < kBlock / 32; ++i) {
    const int c = (threadIdx.x >> 3) + 32 * i, chunk = threadIdx.x & 7;
    const long long row = (long long)tr * kBlock + 16 * chunk;
    if ((long long)tc * kBlock + c >= p.width || row >= p.rows) continue;
    const uint8_t* from = turned + c * kBlock + ((chunk ^ ((c >> 2) & 7)) << 4);
    uint8_t* to = p.yt + ((long long)tc * kBlock + c) * p.ld_yt + row;
    if (vec_t && row + 16 <= p.rows) {
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
    } else {
      for (int e = 0; e < 16 && row + e < p.rows; ++e) to[e] = from[e];
    }
  }
}

template <bool F32, bool VEC>
tsp_status launch(const QuantParams& p, int block, bool vec16, bool vec_t, cudaStream_t s) {
  const long long tiles = ((p.rows + kBlock - 1) / kBlock) * ((p.width + kBlock - 1) / kBlock);
  cudaError_t e;
  if (block == kBlock) {
    e = launch_early(quantize_tile_kernel<F32, true, VEC>, (unsigned)tiles, kThreads, 0, s, p, (int)vec_t);
  } else if (p.yt) {
    e = launch_early(quantize_tile_kernel<F32, false, VEC>, (unsigned)tiles, kThreads, 0, s, p, (int)vec_t);
  } else {
    const long long blocks = p.rows * ((p.width + kBlock - 1) / kBlock);
    const long long per_cta = kThreads / 32 * (vec16 ? 8 : 1);
    const unsigned ctas = (unsigned)((blocks + per_cta - 1) / per_cta);
    if (vec16) e = launch_early(quantize_rows_kernel<F32>, ctas, kThreads, 0, s, p);
    else e = launch_early(quantize_any_rows_kernel<F32>, ctas, kThreads, 0, s, p);
  }
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "quantize: launch");
}

}  // namespace
}  // namespace tsp

using namespace tsp;

extern "C" {

tsp_status tsp_quantize_e4m3(int64_t rows, int64_t width, const void* x, int x_f32, int64_t ld_x, int block,
                             uint8_t* y, int64_t ld_y, float* scales, uint8_t* yt, int64_t ld_yt, float* scales_t,
                             void* stream) {
  TSP_GUARD_BEGIN
  const char* what = "tsp_quantize_e4m3";
  const std::string n(what);
  constexpr int64_t most = (1ll << 31) - 1;
  if (rows < 0 || rows > most || width < 0 || width > most)
    return fail(TSP_ERR_UNSUPPORTED, n + ": rows and width in [0, 2^31) only");
  if (block != 1 && block != kBlock) return fail(TSP_ERR_UNSUPPORTED, n + ": blocks of 1 or 128 rows");
  if (rows == 0 || width == 0) return TSP_OK;
  if ((y == nullptr) != (scales == nullptr) || (yt == nullptr) != (scales_t == nullptr))
    return fail(TSP_ERR_INVALID_ARG, n + ": values and their scales are written together");
  if (!y && !yt) return fail(TSP_ERR_INVALID_ARG, n + ": null output");
  const unsigned es = x_f32 ? 4u : 2u;
  if (!x) return fail(TSP_ERR_INVALID_ARG, n + ": null pointer");
  if (reinterpret_cast<uintptr_t>(x) % es || reinterpret_cast<uintptr_t>(scales) % 4 ||
      reinterpret_cast<uintptr_t>(scales_t) % 4)
    return fail(TSP_ERR_INVALID_ARG, n + ": pointer not aligned to its element");
  if (ld_x < width || (y && ld_y < width) || (yt && ld_yt < rows))
    return fail(TSP_ERR_INVALID_ARG, n + ": row stride below the row's length");
  if (ld_x > (1ll << 40) || ld_y > (1ll << 40) || ld_yt > (1ll << 40))
    return fail(TSP_ERR_UNSUPPORTED, n + ": row stride too large");
  const int64_t groups = (width + kBlock - 1) / kBlock, groups_t = (rows + kBlock - 1) / kBlock;
  // blocks are counted in 32 bits, and a tile is a CTA
  if (rows * groups > most || ((rows + kBlock - 1) / kBlock) * groups > most)
    return fail(TSP_ERR_UNSUPPORTED, n + ": too many blocks");
  const int64_t rs = y ? (block == 1 ? rows : groups_t) * groups * 4 : 0;
  const int64_t ts = yt ? (block == 1 ? width : groups) * groups_t * 4 : 0;
  const Extent all[5] = {extent(x, rows, width * es, ld_x * es), extent(y, y ? rows : 0, width, ld_y), extent(scales, 1, rs, rs),
                         extent(yt, yt ? width : 0, rows, ld_yt), extent(scales_t, 1, ts, ts)};
  for (int i = 1; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlaps(all[i], all[j])) return fail(TSP_ERR_INVALID_ARG, n + ": an output aliases another buffer");
  const QuantParams p{rows, width, x, ld_x, y, ld_y, scales, yt, ld_yt, scales_t};
  // 4 columns at a time where every row of x and y starts on their boundary
  const bool vec = width % 4 == 0 && ld_x % 4 == 0 && reinterpret_cast<uintptr_t>(x) % (4 * es) == 0 &&
                   (!y || (ld_y % 4 == 0 && reinterpret_cast<uintptr_t>(y) % 4 == 0));
  // or, rows alone, 16 bytes of x and as many values of y
  const bool vec16 = width % (16 / es) == 0 && ld_x % (16 / es) == 0 && al16(x) && ld_y % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(y) % 8 == 0;
  const bool vec_t = ld_yt % 16 == 0 && al16(yt);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x_f32) return vec ? launch<true, true>(p, block, vec16, vec_t, s) : launch<true, false>(p, block, vec16, vec_t, s);
  return vec ? launch<false, true>(p, block, vec16, vec_t, s) : launch<false, false>(p, block, vec16, vec_t, s);
  TSP_GUARD_END
}

}  // extern "C"
