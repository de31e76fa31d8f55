// quantize.cu - e4m3 values with an fp32 scale for each block of 128, from bf16 or fp32:
//     scale = max|x| / 448 over the block (1 for zeros, at least 2^-126), q = e4m3(x / scale)
// in the forms that the products of a linear layer read (matmul_e4m3.cu):
//   rows       y  [rows][width]: a scale for 128 columns of one row
//   columns    yt [width][rows]: the transpose, a scale for 128 rows of one column
//   tiles      one scale for 128 x 128 values: y and its transpose hold the same values
//
// Bound: HBM. x is read once, whatever is written. The rows alone are a warp's work each, 128
// columns at a time. What needs a column's largest value or a transpose takes a tile of 128 x 128
// per CTA: each warp holds 16 rows in registers, the columns' maxima meet in shared memory, and
// the transposed bytes go through a 16 KB tile there (16-byte chunks, swizzled by their column) so
// that both layouts are written in runs of 128 bytes.
#include "e4m3.cuh"
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

// Four columns c to c + 3 of a row (zeros behind the width).
template <bool F32, bool VEC>
__device__ __forceinline__ void load4(const void* x, long long at, long long left, float (&v)[4]) {
  if constexpr (VEC) {
    if (left <= 0) {
      v[0] = v[1] = v[2] = v[3] = 0.f;
    } else if constexpr (F32) {
      const float4 u = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(x) + at));
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x) + at));
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = 0.f;
      if (e < left)
        v[e] = F32 ? static_cast<const float*>(x)[at + e] : __bfloat162float(static_cast<const __nv_bfloat16*>(x)[at + e]);
    }
  }
}

__device__ __forceinline__ uint32_t quantize4(const Quotient& by, const float (&v)[4]) {
  float a = v[0], b = v[1], c = v[2], d = v[3];
  by.pair(a, b);
  by.pair(c, d);
  return to_e4m3x4(a, b, c, d);
}

template <bool VEC>
__device__ __forceinline__ void store4(uint8_t* y, long long left, uint32_t q) {
  if constexpr (VEC) {
    if (left > 0) *reinterpret_cast<uint32_t*>(y) = q;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) y[e] = (uint8_t)(q >> (8 * e));
  }
}

// One warp per row and 128 columns, four of them at a time. VEC: the width is a multiple of 4 and
// every row starts on 16 (fp32) or 8 (bf16) bytes, in y on 4.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantParams p) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  const long long groups = (p.width + kBlock - 1) / kBlock;
  const long long blocks = p.rows * groups;
  const long long first = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * U;
  dependents_may_start();
  prior_kernel_done();
  float v[U][4];
  long long row[U], left[U];
  int group[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const long long b = first + i;
    row[i] = b / groups;
    group[i] = (int)(b - row[i] * groups);
    const long long col = (long long)group[i] * kBlock + 4 * lane;
    left[i] = b < blocks ? p.width - col : 0;
    load4<F32, VEC>(p.x, row[i] * p.ld_x + col, left[i], v[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (first + i >= blocks) break;
    const uint32_t top = __reduce_max_sync(
        0xffffffffu, max(max(magnitude(v[i][0]), magnitude(v[i][1])), max(magnitude(v[i][2]), magnitude(v[i][3]))));
    const float scale = e4m3_scale(top);
    if (lane == 0) p.scales[first + i] = scale;
    store4<VEC>(p.y + row[i] * p.ld_y + (long long)group[i] * kBlock + 4 * lane, left[i], quantize4(Quotient(scale), v[i]));
  }
}

// One CTA per tile of 128 x 128. TILE: one scale for all of it. VEC as above; VEC_T: yt's rows start
// on 16 bytes.
template <bool F32, bool TILE, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) quantize_tile_kernel(const QuantParams p, int vec_t) {
  __shared__ __align__(16) uint8_t turned[kBlock * kBlock];
  __shared__ __align__(16) uint32_t tops[kThreads / 32][kBlock];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tiles_w = (p.width + kBlock - 1) / kBlock, tiles_r = (p.rows + kBlock - 1) / kBlock;
  const long long tr = blockIdx.x / tiles_w, tc = blockIdx.x - tr * tiles_w;
  const long long row0 = tr * kBlock + 16 * warp, col = tc * kBlock + 4 * lane;
  dependents_may_start();
  prior_kernel_done();
  float v[16][4];
#pragma unroll
  for (int r = 0; r < 16; ++r)
    load4<F32, VEC>(p.x, (row0 + r) * p.ld_x + col, row0 + r < p.rows ? p.width - col : 0, v[r]);

  uint32_t top[4] = {0u, 0u, 0u, 0u};  // of this lane's columns over this warp's rows
#pragma unroll
  for (int r = 0; r < 16; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e] = max(top[e], magnitude(v[r][e]));
  if constexpr (TILE) {
    const uint32_t t = __reduce_max_sync(0xffffffffu, max(max(top[0], top[1]), max(top[2], top[3])));
    if (lane == 0) tops[0][warp] = t;
    __syncthreads();
    const float scale = e4m3_scale(__reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? tops[0][lane] : 0u));
    const Quotient by(scale);
    if (threadIdx.x == 0) {
      if (p.y) p.scales[tr * tiles_w + tc] = scale;
      if (p.yt) p.scales_t[tc * tiles_r + tr] = scale;
    }
    uint32_t q[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      q[r] = quantize4(by, v[r]);
      if (p.y && row0 + r < p.rows) store4<VEC>(p.y + (row0 + r) * p.ld_y + col, p.width - col, q[r]);
    }
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
    if (p.y) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (row0 + r >= p.rows) break;
        const uint32_t t = __reduce_max_sync(
            0xffffffffu, max(max(magnitude(v[r][0]), magnitude(v[r][1])), max(magnitude(v[r][2]), magnitude(v[r][3]))));
        const float scale = e4m3_scale(t);
        if (lane == 0) p.scales[(row0 + r) * tiles_w + tc] = scale;
        store4<VEC>(p.y + (row0 + r) * p.ld_y + col, p.width - col, quantize4(Quotient(scale), v[r]));
      }
    }
    *reinterpret_cast<uint4*>(&tops[warp][4 * lane]) = make_uint4(top[0], top[1], top[2], top[3]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      const uint4 t = *reinterpret_cast<const uint4*>(&tops[k][4 * lane]);
      top[0] = max(top[0], t.x), top[1] = max(top[1], t.y), top[2] = max(top[2], t.z), top[3] = max(top[3], t.w);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float scale = e4m3_scale(top[e]);
      const Quotient by(scale);
      if (warp == 0 && col + e < p.width) p.scales_t[(col + e) * tiles_r + tr] = scale;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float four[4] = {v[4 * k][e], v[4 * k + 1][e], v[4 * k + 2][e], v[4 * k + 3][e]};
        w[k] = quantize4(by, four);
      }
      *reinterpret_cast<uint4*>(turned + (4 * lane + e) * kBlock + ((warp ^ (lane & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __syncthreads();
  // 16 rows of x of one column per thread and step
#pragma unroll
  for (int i = 0; i < kBlock / 32; ++i) {
    const int c = (threadIdx.x >> 3) + 32 * i, chunk = threadIdx.x & 7;
    const long long row = tr * kBlock + 16 * chunk;
    if (tc * kBlock + c >= p.width || row >= p.rows) continue;
    const uint8_t* from = turned + c * kBlock + ((chunk ^ ((c >> 2) & 7)) << 4);
    uint8_t* to = p.yt + (tc * kBlock + c) * p.ld_yt + row;
    if (vec_t && row + 16 <= p.rows) {
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
    } else {
      for (int e = 0; e < 16 && row + e < p.rows; ++e) to[e] = from[e];
    }
  }
}

template <bool F32, bool VEC>
tsp_status launch(const QuantParams& p, int block, bool vec_t, cudaStream_t s) {
  const long long tiles = ((p.rows + kBlock - 1) / kBlock) * ((p.width + kBlock - 1) / kBlock);
  cudaError_t e;
  if (block == kBlock) {
    e = launch_early(quantize_tile_kernel<F32, true, VEC>, (unsigned)tiles, kThreads, 0, s, p, (int)vec_t);
  } else if (p.yt) {
    e = launch_early(quantize_tile_kernel<F32, false, VEC>, (unsigned)tiles, kThreads, 0, s, p, (int)vec_t);
  } else {
    const long long per_cta = kThreads / 32 * 4;
    const long long ctas = (p.rows * ((p.width + kBlock - 1) / kBlock) + per_cta - 1) / per_cta;
    e = launch_early(quantize_rows_kernel<F32, VEC>, (unsigned)ctas, kThreads, 0, s, p);
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
  if (x == y || x == yt || (y && y == yt) || (scales && scales == scales_t))
    return fail(TSP_ERR_INVALID_ARG, n + ": an output aliases another buffer");
  // one CTA per 32 groups of a row, or per tile
  const int64_t groups = (width + kBlock - 1) / kBlock;
  if (rows * groups > 32 * most || ((rows + kBlock - 1) / kBlock) * groups > most)
    return fail(TSP_ERR_UNSUPPORTED, n + ": too many blocks");
  const QuantParams p{rows, width, x, ld_x, y, ld_y, scales, yt, ld_yt, scales_t};
  // 4 columns at a time where every row of x and y starts on their boundary
  const bool vec = width % 4 == 0 && ld_x % 4 == 0 && reinterpret_cast<uintptr_t>(x) % (4 * es) == 0 &&
                   (!y || (ld_y % 4 == 0 && reinterpret_cast<uintptr_t>(y) % 4 == 0));
  const bool vec_t = ld_yt % 16 == 0 && al16(yt);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x_f32) return vec ? launch<true, true>(p, block, vec_t, s) : launch<true, false>(p, block, vec_t, s);
  return vec ? launch<false, true>(p, block, vec_t, s) : launch<false, false>(p, block, vec_t, s);
  TSP_GUARD_END
}

}  // extern "C"
