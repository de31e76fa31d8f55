// rmsnorm.cu - root-mean-square norm with the residual's addition, forward (bf16 or
// e4m3 output) and backward: the step between two blocks of a pre-norm stack.
//
// Forward, per row of `width` elements (sums in fp32):
//     h = x + r            stored in r's type (bf16 or fp32); h = x without a residual
//     y = h * rstd * w,    rstd = 1 / sqrt(mean(h^2) + eps), from the unrounded h
//     e4m3: per row or per 128 columns  scale = max|y| / 448,  y8 = e4m3(y / scale)
// Backward, with g = dy * w and n = width:
//     dx = rstd * g - h * rstd^3 * (sum(g h) / n)  (+ dh)
//     dw = sum over rows of dy * h * rstd
// rstd is taken again from h: the row is in registers for sum(g h) in any case, so a
// saved rstd would only add traffic.
//
// Bound: HBM. A row is read once, stays in registers between its reduction and its
// outputs, and is written once. Layout of the work: a row of up to 1024 elements per
// warp (no block barrier), a longer one per CTA; each thread owns the same columns of
// every row it meets, so the weight is loaded once and dw is summed in registers.
// CTAs are persistent.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "tsp_device.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace {

enum { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };
constexpr float kE4m3Max = 448.0f;
constexpr int kMaxWidth = 32768;
// CTAs of the backward at most: three per SM of this part, a constant so that the order
// of dw's sum is the same on every device
constexpr int kBwdCtas = 456;

// VEC consecutive elements as fp32. VEC is 8 (16-byte loads) or 1.
template <int VEC>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    v[0] = __bfloat162float(*p);
  }
}

template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}

template <int VEC>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    uint4 u;
    u.x = pack_bf16x2(v[0], v[1]);
    u.y = pack_bf16x2(v[2], v[3]);
    u.z = pack_bf16x2(v[4], v[5]);
    u.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

template <int VEC>
__device__ __forceinline__ void store_f32(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}

// An element range of a stream kept in bf16 or fp32.
template <int VEC, int RES>
__device__ __forceinline__ void load_stream(const void* p, long long i, float (&v)[VEC]) {
  if constexpr (RES == RES_F32) load_f32<VEC>(static_cast<const float*>(p) + i, v);
  else load_bf16<VEC>(static_cast<const __nv_bfloat16*>(p) + i, v);
}
template <int VEC, int RES>
__device__ __forceinline__ void store_stream(void* p, long long i, const float (&v)[VEC]) {
  if constexpr (RES == RES_F32) store_f32<VEC>(static_cast<float*>(p) + i, v);
  else store_bf16<VEC>(static_cast<__nv_bfloat16*>(p) + i, v);
}

// Sum over the row's threads, the same bits in every thread. WARP: the row's threads are
// one warp. Otherwise the whole block, through `part` (one float per warp); the caller
// alternates between two such arrays, so one barrier per reduction is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Largest bit pattern of non-negative floats: NaN above infinity above the numbers.
template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    v = __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0u);
  }
  return v;
}

// The scale of a group whose largest |y| has the bits `top`. A group of zeros takes 1;
// the smallest scale is the smallest normal number, so that its reciprocal is finite.
// NaN or infinity in the group gives a NaN or infinite scale.
__device__ __forceinline__ float e4m3_scale(uint32_t top) {
  const float t = __uint_as_float(top);
  if (top == 0u) return 1.f;
  if (top > 0x7f800000u) return t;
  return fmaxf(t / kE4m3Max, 1.17549435e-38f);
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
// four values, the first in the low byte: one conversion instruction per pair
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

struct NormParams {
  const __nv_bfloat16* x;
  const void* r;
  const __nv_bfloat16* w;
  void* h;
  void* y;        // bf16 or e4m3
  float* scales;
  long long rows;
  int width;
  int group;      // e4m3: 128, or 0 for one scale per row
  float eps;
};

// One row per warp (WARP) or per CTA; NV times VEC elements per thread.
// MAXT: the largest block, which bounds the registers of a thread.
template <int VEC, int NV, bool WARP, int RES, bool E4M3, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_fwd_kernel(const NormParams p) {
  __shared__ float part[2][32];
  __shared__ uint32_t tops[2][VEC == 1 && E4M3 ? kMaxWidth / 128 : 32];
  const int lanes = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const long long row0 = WARP ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const long long step = (long long)gridDim.x * (WARP ? 4 : 1);
  const float inv_n = 1.f / (float)p.width;
  float w[NV][VEC], v[NV][VEC];
  auto col = [&](int i) { return (i * lanes + tid) * VEC; };
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (c < p.width) {
        load_bf16<VEC>(p.x + row * p.width + c, v[i]);
        if constexpr (RES != RES_NONE) {
          float r[VEC];
          load_stream<VEC, RES>(p.r, row * p.width + c, r);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += r[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < p.width) load_bf16<VEC>(p.w + col(i), w[i]);
  int odd = 0;
  for (long long row = row0; row < p.rows; row += step, odd ^= 1) {
    load(row);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    const float rstd = 1.f / sqrtf(row_sum<WARP>(ss, part[odd]) * inv_n + p.eps);
    if constexpr (RES != RES_NONE) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < p.width) store_stream<VEC, RES>(p.h, row * p.width + col(i), v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = col(i) < p.width ? v[i][e] * rstd * w[i][e] : 0.f;
    }
    if constexpr (!E4M3) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < p.width)
          store_bf16<VEC>(static_cast<__nv_bfloat16*>(p.y) + row * p.width + col(i), v[i]);
    } else {
      uint8_t* y8 = static_cast<uint8_t*>(p.y) + row * p.width;
      auto top_of = [&](int i) {
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) t = max(t, __float_as_uint(fabsf(v[i][e])));
        return t;
      };
      auto store8 = [&](int i, float scale) {
        const float inv = 1.f / scale;
        if constexpr (VEC == 8) {
          *reinterpret_cast<uint2*>(y8 + col(i)) =
              make_uint2(to_e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                         to_e4m3x4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv));
        } else {
          y8[col(i)] = to_e4m3(v[i][0] * inv);
        }
      };
      if (p.group == 0) {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) t = max(t, top_of(i));
        const float scale = e4m3_scale(row_max<WARP>(t, tops[odd]));
        if (tid == 0) p.scales[row] = scale;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < p.width) store8(i, scale);
      } else if constexpr (VEC == 8) {
        // 16 consecutive threads hold 128 consecutive columns
        const int groups = (p.width + 127) / 128;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint32_t t = top_of(i);
#pragma unroll
          for (int o = 8; o; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
          const float scale = e4m3_scale(t);
          if (col(i) < p.width) {
            if ((tid & 15) == 0) p.scales[row * groups + col(i) / 128] = scale;
            store8(i, scale);
          }
        }
      } else {
        // 128 consecutive threads hold a group: the largest through shared memory (a
        // maximum does not depend on the order of the atomics)
        const int groups = (p.width + 127) / 128;
        __syncthreads();
        for (int g = threadIdx.x; g < groups; g += blockDim.x) tops[0][g] = 0u;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < p.width) atomicMax(&tops[0][col(i) / 128], top_of(i));
        __syncthreads();
        for (int g = threadIdx.x; g < groups; g += blockDim.x)
          p.scales[row * groups + g] = e4m3_scale(tops[0][g]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < p.width) store8(i, e4m3_scale(tops[0][col(i) / 128]));
      }
    }
  }
}

// Longer rows, staged in shared memory: each thread copies its own 16-byte pieces of the
// rows ahead (cp.async) and later reads only those, so a wait for its own copies is all the
// ordering that is needed, and STAGES - 1 rows of every CTA are in flight under the
// arithmetic and the barriers of the current one.
__device__ __forceinline__ void copy_ahead(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(global) : "memory");
}

template <int RES, bool E4M3, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 4 : 1) rmsnorm_fwd_ring_kernel(const NormParams p) {
  constexpr int NV = 2;
  constexpr int SP = RES == RES_NONE ? 0 : RES == RES_F32 ? 2 : 1;  // 16-byte pieces of 8 stream elements
  constexpr int PIECES = NV * (1 + SP);
  extern __shared__ uint4 ring[];  // [STAGES][PIECES][threads]
  __shared__ float part[2][32];
  __shared__ uint32_t tops[2][32];
  const int tid = threadIdx.x, lanes = blockDim.x;
  const float inv_n = 1.f / (float)p.width;
  auto col = [&](int i) { return (i * lanes + tid) * 8; };
  auto slot = [&](int stage, int piece) { return ring + (stage * PIECES + piece) * lanes + tid; };
  auto fetch = [&](long long row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) >= p.width) continue;
        const long long at = row * p.width + col(i);
        copy_ahead(slot(stage, i), p.x + at);
#pragma unroll
        for (int u = 0; u < SP; ++u)
          copy_ahead(slot(stage, NV + i * SP + u),
                     static_cast<const char*>(p.r) + at * (RES == RES_F32 ? 4 : 2) + 16 * u);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
  uint4 w[NV];  // bf16: unpacked where it is used
#pragma unroll
  for (int i = 0; i < NV; ++i)
    w[i] = col(i) < p.width ? *reinterpret_cast<const uint4*>(p.w + col(i)) : make_uint4(0u, 0u, 0u, 0u);
  int odd = 0, stage = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, odd ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) < p.width) {
        load_bf16<8>(reinterpret_cast<const __nv_bfloat16*>(slot(stage, i)), v[i]);
        if constexpr (RES != RES_NONE) {
          float r[8];
          if constexpr (RES == RES_F32) {
            const float4 a = *reinterpret_cast<const float4*>(slot(stage, NV + i * SP));
            const float4 b = *reinterpret_cast<const float4*>(slot(stage, NV + i * SP + 1));
            r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
            r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
          } else {
            load_bf16<8>(reinterpret_cast<const __nv_bfloat16*>(slot(stage, NV + i * SP)), r);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += r[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    // this stage is read; the one before it takes the row furthest ahead
    fetch(row + (long long)(STAGES - 1) * gridDim.x, stage == 0 ? STAGES - 1 : stage - 1);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    const float rstd = 1.f / sqrtf(row_sum<false>(ss, part[odd]) * inv_n + p.eps);
    if constexpr (RES != RES_NONE) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < p.width) store_stream<8, RES>(p.h, row * p.width + col(i), v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[i][2 * e] *= rstd * bf16_lo(u[e]);
        v[i][2 * e + 1] *= rstd * bf16_hi(u[e]);
      }
    }
    if constexpr (!E4M3) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < p.width)
          store_bf16<8>(static_cast<__nv_bfloat16*>(p.y) + row * p.width + col(i), v[i]);
    } else {
      uint8_t* y8 = static_cast<uint8_t*>(p.y) + row * p.width;
      uint32_t top[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        top[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top[i] = max(top[i], __float_as_uint(fabsf(v[i][e])));
      }
      if (p.group == 0) {
        const uint32_t t = row_max<false>(max(top[0], top[1]), tops[odd]);
        top[0] = top[1] = t;
        if (tid == 0) p.scales[row] = e4m3_scale(t);
      } else {
        // 16 consecutive threads hold 128 consecutive columns
        const int groups = (p.width + 127) / 128;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int o = 8; o; o >>= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
          if (col(i) < p.width && (tid & 15) == 0) p.scales[row * groups + col(i) / 128] = e4m3_scale(top[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float inv = 1.f / e4m3_scale(top[i]);
        if (col(i) < p.width)
          *reinterpret_cast<uint2*>(y8 + col(i)) =
              make_uint2(to_e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                         to_e4m3x4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv));
      }
    }
  }
}

struct NormBwdParams {
  const void* h;
  const __nv_bfloat16* w;
  const __nv_bfloat16* dy;
  const void* dh;  // optional, h's type
  void* dx;        // h's type
  __nv_bfloat16* dx16;  // optional
  float* partial;  // [CTAs][width]
  long long rows;
  int width;
  float eps;
};

// One row per CTA at a time; dw of the CTA's rows in registers, written as one partial row.
template <int VEC, int NV, int RES>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_kernel(const NormBwdParams p) {
  __shared__ float part[2][2][32];
  const int tid = threadIdx.x, lanes = blockDim.x;
  const float inv_n = 1.f / (float)p.width;
  auto col = [&](int i) { return (i * lanes + tid) * VEC; };
  float w[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = 0.f;
    if (col(i) < p.width) load_bf16<VEC>(p.w + col(i), w[i]);
  }
  int odd = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, odd ^= 1) {
    float h[NV][VEC], g[NV][VEC];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (c < p.width) {
        load_stream<VEC, RES>(p.h, row * p.width + c, h[i]);
        load_bf16<VEC>(p.dy + row * p.width + c, g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[i][e] = g[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        ss = fmaf(h[i][e], h[i][e], ss);
        sg = fmaf(g[i][e] * w[i][e], h[i][e], sg);
      }
    }
    // both sums behind one barrier
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    if ((tid & 31) == 0) {
      part[odd][0][tid >> 5] = ss;
      part[odd][1][tid >> 5] = sg;
    }
    __syncthreads();
    const bool in = (tid & 31) < (lanes >> 5);
    ss = in ? part[odd][0][tid & 31] : 0.f;
    sg = in ? part[odd][1][tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    const float rstd = 1.f / sqrtf(ss * inv_n + p.eps);
    const float coef = rstd * rstd * (sg * inv_n);  // dx = rstd (g - h coef)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (c >= p.width) continue;
      float d[VEC];
      if (p.dh != nullptr) load_stream<VEC, RES>(p.dh, row * p.width + c, d);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float t = rstd * (g[i][e] * w[i][e] - h[i][e] * coef);
        dw[i][e] = fmaf(g[i][e], h[i][e] * rstd, dw[i][e]);
        d[e] = p.dh != nullptr ? d[e] + t : t;
      }
      store_stream<VEC, RES>(p.dx, row * p.width + c, d);
      if (p.dx16 != nullptr) store_bf16<VEC>(p.dx16 + row * p.width + c, d);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < p.width) store_f32<VEC>(p.partial + (long long)blockIdx.x * p.width + col(i), dw[i]);
}

// The same with the rows staged in shared memory, as in the forward's ring kernel.
template <int NV, int RES, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_bwd_ring_kernel(const NormBwdParams p) {
  constexpr int SP = RES == RES_F32 ? 2 : 1;  // 16-byte pieces of 8 stream elements
  extern __shared__ uint4 ring[];             // [STAGES][pieces][threads]
  __shared__ float part[2][2][32];
  const int tid = threadIdx.x, lanes = blockDim.x;
  const bool has_dh = p.dh != nullptr;
  const int pieces = NV * (SP + 1 + (has_dh ? SP : 0));
  const float inv_n = 1.f / (float)p.width;
  auto col = [&](int i) { return (i * lanes + tid) * 8; };
  auto slot = [&](int stage, int piece) { return ring + ((long long)stage * pieces + piece) * lanes + tid; };
  const size_t es = RES == RES_F32 ? 4 : 2;
  auto fetch = [&](long long row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) >= p.width) continue;
        const long long at = row * p.width + col(i);
        const char* h = static_cast<const char*>(p.h) + at * es;
        const char* d = static_cast<const char*>(p.dh) + at * es;
#pragma unroll
        for (int u = 0; u < SP; ++u) {
          copy_ahead(slot(stage, i * SP + u), h + 16 * u);
          if (has_dh) copy_ahead(slot(stage, NV * (SP + 1) + i * SP + u), d + 16 * u);
        }
        copy_ahead(slot(stage, NV * SP + i), p.dy + at);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto stream_of = [&](int stage, int piece, float (&v)[8]) {
    if constexpr (RES == RES_F32) {
      const float4 a = *reinterpret_cast<const float4*>(slot(stage, piece));
      const float4 b = *reinterpret_cast<const float4*>(slot(stage, piece + 1));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      load_bf16<8>(reinterpret_cast<const __nv_bfloat16*>(slot(stage, piece)), v);
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = dw[i][e] = 0.f;
    if (col(i) < p.width) load_bf16<8>(p.w + col(i), w[i]);
  }
  int odd = 0, stage = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, odd ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    float h[NV][8], g[NV][8];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) < p.width) {
        stream_of(stage, i * SP, h[i]);
        load_bf16<8>(reinterpret_cast<const __nv_bfloat16*>(slot(stage, NV * SP + i)), g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = g[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(h[i][e], h[i][e], ss);
        sg = fmaf(g[i][e] * w[i][e], h[i][e], sg);
      }
    }
    // the stage of the row before is read to its end: the row furthest ahead goes there
    {
      const int into = stage == 0 ? STAGES - 1 : stage - 1;
      fetch(row + (long long)(STAGES - 1) * gridDim.x, into);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    if ((tid & 31) == 0) {
      part[odd][0][tid >> 5] = ss;
      part[odd][1][tid >> 5] = sg;
    }
    __syncthreads();
    const bool in = (tid & 31) < (lanes >> 5);
    ss = in ? part[odd][0][tid & 31] : 0.f;
    sg = in ? part[odd][1][tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    const float rstd = 1.f / sqrtf(ss * inv_n + p.eps);
    const float coef = rstd * rstd * (sg * inv_n);  // dx = rstd (g - h coef)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (c >= p.width) continue;
      float d[8];
      if (has_dh) stream_of(stage, NV * (SP + 1) + i * SP, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = rstd * (g[i][e] * w[i][e] - h[i][e] * coef);
        dw[i][e] = fmaf(g[i][e], h[i][e] * rstd, dw[i][e]);
        d[e] = has_dh ? d[e] + t : t;
      }
      store_stream<8, RES>(p.dx, row * p.width + c, d);
      if (p.dx16 != nullptr) store_bf16<8>(p.dx16 + row * p.width + c, d);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < p.width) store_f32<8>(p.partial + (long long)blockIdx.x * p.width + col(i), dw[i]);
}

// dw[c] = sum of the partial rows, in a fixed order: 32 row groups per column, then their
// sum.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* __restrict__ partial, int n,
                                                          int width, float* __restrict__ dw) {
  __shared__ float part[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.f;
  if (c < width)
    for (int r = ry; r < n; r += 32) s += partial[(long long)r * width + c];
  part[ry][cx] = s;
  __syncthreads();
  // column ry's 32 sums, one per lane
  s = part[cx][ry];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (cx == 0 && blockIdx.x * 32 + ry < width) dw[blockIdx.x * 32 + ry] = s;
}

bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (!al16(q)) return false;
  return true;
}

// Threads of a CTA that holds a row of `items` (vectors or elements), NV per thread.
int row_threads(int items, int nv) { return ((items + nv - 1) / nv + 31) / 32 * 32; }

template <int VEC, int NV, bool WARP, int RES, bool E4M3>
void launch_fwd_variant(const NormParams& p, cudaStream_t s) {
  constexpr int MAXT = WARP ? 128 : 1024;
  const int threads = WARP ? 128 : row_threads((p.width + VEC - 1) / VEC, NV);
  const long long blocks = WARP ? (p.rows + 3) / 4 : p.rows;
  // resident CTAs: 2048 threads per SM
  const long long cap = (long long)sm_count() * std::max(1, 2048 / threads);
  rmsnorm_fwd_kernel<VEC, NV, WARP, RES, E4M3, MAXT>
      <<<(unsigned)std::min(blocks, cap), threads, 0, s>>>(p);
}

template <int RES, bool E4M3, int STAGES, int MAXT>
tsp_status launch_fwd_ring(const NormParams& p, int threads, cudaStream_t s) {
  auto kernel = rmsnorm_fwd_ring_kernel<RES, E4M3, STAGES, MAXT>;
  const size_t smem = (size_t)STAGES * 2 * (1 + (RES == RES_NONE ? 0 : RES == RES_F32 ? 2 : 1)) * 16 * threads;
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                            "rmsnorm: cudaFuncSetAttribute"));
  // resident CTAs: by registers (four of 256 threads, one of 1024) and by shared memory
  const long long per_sm = std::min<long long>(std::max(1, 1024 / threads), (220 * 1024) / (long long)smem);
  const long long cap = (long long)sm_count() * std::max<long long>(1, per_sm);
  kernel<<<(unsigned)std::min<long long>(p.rows, cap), threads, smem, s>>>(p);
  return TSP_OK;
}

template <int RES, bool E4M3>
tsp_status launch_fwd_res(const NormParams& p, bool vec, cudaStream_t s) {
  if (vec) {
    const int vecs = p.width / 8;
    const int threads = row_threads(vecs, 2);
    if (vecs <= 32) launch_fwd_variant<8, 1, true, RES, E4M3>(p, s);
    else if (vecs <= 64) launch_fwd_variant<8, 2, true, RES, E4M3>(p, s);
    else if (vecs <= 128) launch_fwd_variant<8, 4, true, RES, E4M3>(p, s);
    else if (threads <= 256) return launch_fwd_ring<RES, E4M3, 3, 256>(p, threads, s);
    else if (threads <= 1024) return launch_fwd_ring<RES, E4M3, 2, 1024>(p, threads, s);
    else launch_fwd_variant<8, 4, false, RES, E4M3>(p, s);
  } else {
    if (p.width <= 4096) launch_fwd_variant<1, 8, false, RES, E4M3>(p, s);
    else launch_fwd_variant<1, 32, false, RES, E4M3>(p, s);
  }
  return TSP_OK;
}

tsp_status launch_fwd(const NormParams& p, int res, bool e4m3, bool vec, cudaStream_t s) {
  if (p.rows == 0) return TSP_OK;
  tsp_status st;
  if (e4m3) {
    st = res == RES_NONE ? launch_fwd_res<RES_NONE, true>(p, vec, s)
         : res == RES_BF16 ? launch_fwd_res<RES_BF16, true>(p, vec, s)
                           : launch_fwd_res<RES_F32, true>(p, vec, s);
  } else {
    st = res == RES_NONE ? launch_fwd_res<RES_NONE, false>(p, vec, s)
         : res == RES_BF16 ? launch_fwd_res<RES_BF16, false>(p, vec, s)
                           : launch_fwd_res<RES_F32, false>(p, vec, s);
  }
  if (st != TSP_OK) return st;
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "rmsnorm: launch");
}

template <int VEC, int NV, int RES>
void launch_bwd_variant(const NormBwdParams& p, int ctas, cudaStream_t s) {
  rmsnorm_bwd_kernel<VEC, NV, RES>
      <<<ctas, row_threads((p.width + VEC - 1) / VEC, NV), 0, s>>>(p);
}

template <int NV, int RES, int STAGES, int MAXT>
tsp_status launch_bwd_ring(const NormBwdParams& p, int ctas, int threads, size_t smem, cudaStream_t s) {
  auto kernel = rmsnorm_bwd_ring_kernel<NV, RES, STAGES, MAXT>;
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                            "rmsnorm backward: cudaFuncSetAttribute"));
  kernel<<<ctas, threads, smem, s>>>(p);
  return TSP_OK;
}

template <int RES>
tsp_status launch_bwd_res(const NormBwdParams& p, bool vec, int ctas, cudaStream_t s) {
  if (!vec) {
    if (p.width <= 4096) launch_bwd_variant<1, 8, RES>(p, ctas, s);
    else launch_bwd_variant<1, 32, RES>(p, ctas, s);
    return TSP_OK;
  }
  const int vecs = p.width / 8;
  const int nv = vecs <= 128 ? 1 : 2;
  const int threads = row_threads(vecs, nv);
  // shared memory of a staged row: whole 16-byte pieces of every thread
  const size_t row = (size_t)threads * nv * 16 * ((RES == RES_F32 ? 2 : 1) * (p.dh ? 2 : 1) + 1);
  // three stages where three CTAs fit an SM with them, else two; a row too wide for two
  // stages is loaded straight into registers
  const bool three = 3 * row <= 74 * 1024;
  const size_t smem = (three ? 3 : 2) * row;
  if (threads <= 1024 && smem <= 220 * 1024) {
    if (nv == 1) return launch_bwd_ring<1, RES, 3, 256>(p, ctas, threads, 3 * row, s);
    if (threads <= 256) {
      if (three) return launch_bwd_ring<2, RES, 3, 256>(p, ctas, threads, smem, s);
      return launch_bwd_ring<2, RES, 2, 256>(p, ctas, threads, smem, s);
    }
    return launch_bwd_ring<2, RES, 2, 1024>(p, ctas, threads, 2 * row, s);
  }
  launch_bwd_variant<8, 4, RES>(p, ctas, s);
  return TSP_OK;
}

// Checks shared by the three calls.
tsp_status check_shape(const char* what, int64_t rows, int width, float eps) {
  const std::string n(what);
  if (rows < 0 || rows > (1ll << 31) - 1 || width < 1 || width > kMaxWidth)
    return fail(TSP_ERR_UNSUPPORTED, n + ": rows in [0, 2^31) and width in [1, 32768] only");
  if (!(eps > 0.f) || !std::isfinite(eps))
    return fail(TSP_ERR_INVALID_ARG, n + ": eps must be positive and finite");
  return TSP_OK;
}
tsp_status check_natural(const char* what, const void* ptr, unsigned align, bool optional) {
  if (!ptr && optional) return TSP_OK;
  if (!ptr) return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": null pointer");
  if (reinterpret_cast<uintptr_t>(ptr) % align)
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": pointer not aligned to its element");
  return TSP_OK;
}

tsp_status rmsnorm_fwd(const char* what, int64_t rows, int width, const void* x, const void* r,
                       int r_f32, const void* w, float eps, void* h, void* y, bool e4m3, int group,
                       float* scales, cudaStream_t s) {
  TSP_TRY(check_shape(what, rows, width, eps));
  if (rows == 0) return TSP_OK;
  const unsigned rs = r_f32 ? 4u : 2u;
  TSP_TRY(check_natural(what, x, 2, false));
  TSP_TRY(check_natural(what, w, 2, false));
  TSP_TRY(check_natural(what, y, e4m3 ? 1u : 2u, false));
  TSP_TRY(check_natural(what, r, rs, true));
  TSP_TRY(check_natural(what, h, rs, true));
  if ((r == nullptr) != (h == nullptr))
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": h is written with a residual and only then");
  if (e4m3) TSP_TRY(check_natural(what, scales, 4, false));
  if (y == r || y == h)
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": y aliases the residual stream");
  if (x == h || (e4m3 && x == y) || (x == r && r == h))
    return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": x aliases an output");
  NormParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.r = r;
  p.w = static_cast<const __nv_bfloat16*>(w);
  p.h = h;
  p.y = y;
  p.scales = scales;
  p.rows = rows;
  p.width = width;
  p.group = group;
  p.eps = eps;
  // 16-byte loads where every row of every buffer starts on 16 bytes (8 for the e4m3
  // rows, which then follow); single elements otherwise
  const bool vec = width % 8 == 0 && aligned16({x, r, w, h, y});
  return launch_fwd(p, r == nullptr ? RES_NONE : r_f32 ? RES_F32 : RES_BF16, e4m3, vec, s);
}

}  // namespace
}  // namespace tsp

using namespace tsp;

extern "C" {

tsp_status tsp_rmsnorm_fwd(int64_t rows, int width, const tsp_bf16* x, const void* residual,
                           int residual_f32, const tsp_bf16* weight, float eps, void* h, tsp_bf16* y,
                           void* stream) {
  return rmsnorm_fwd("tsp_rmsnorm_fwd", rows, width, x, residual, residual_f32, weight, eps, h, y,
                     false, 0, nullptr, static_cast<cudaStream_t>(stream));
}

tsp_status tsp_rmsnorm_fwd_e4m3(int64_t rows, int width, const tsp_bf16* x, const void* residual,
                                int residual_f32, const tsp_bf16* weight, float eps, int group,
                                void* h, uint8_t* y, float* scales, void* stream) {
  if (group != 0 && group != 128)
    return fail(TSP_ERR_UNSUPPORTED, "tsp_rmsnorm_fwd_e4m3: group 0 (a row) or 128 columns");
  return rmsnorm_fwd("tsp_rmsnorm_fwd_e4m3", rows, width, x, residual, residual_f32, weight, eps, h,
                     y, true, group, scales, static_cast<cudaStream_t>(stream));
}

size_t tsp_rmsnorm_workspace_bytes(int64_t rows, int width) {
  if (rows < 0 || width < 1 || width > kMaxWidth) return 0;
  const int64_t ctas = rows < kBwdCtas ? (rows < 1 ? 1 : rows) : kBwdCtas;
  return align256((size_t)ctas * (size_t)width * sizeof(float));
}

tsp_status tsp_rmsnorm_bwd(int64_t rows, int width, const void* h, int h_f32, const tsp_bf16* weight,
                           float eps, const tsp_bf16* dy, const void* dh, void* dx, tsp_bf16* dx16,
                           float* dw, void* ws, void* stream) {
  const char* what = "tsp_rmsnorm_bwd";
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TSP_TRY(check_shape(what, rows, width, eps));
  TSP_TRY(check_natural(what, dw, 4, false));
  TSP_TRY(check_ws(ws, what));
  if (rows == 0) {
    cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)width * sizeof(float), s);
    return e == cudaSuccess ? TSP_OK : cuda_fail(e, what);
  }
  const unsigned hs = h_f32 ? 4u : 2u;
  TSP_TRY(check_natural(what, h, hs, false));
  TSP_TRY(check_natural(what, dx, hs, false));
  TSP_TRY(check_natural(what, dh, hs, true));
  TSP_TRY(check_natural(what, weight, 2, false));
  TSP_TRY(check_natural(what, dy, 2, false));
  TSP_TRY(check_natural(what, dx16, 2, true));
  const void* d16 = dx16;
  if (dx == h || (d16 && (d16 == h || d16 == dx || d16 == dh)) || (h_f32 && dx == dy))
    return fail(TSP_ERR_INVALID_ARG, "tsp_rmsnorm_bwd: an output aliases h or another output");
  NormBwdParams p{};
  p.h = h;
  p.w = reinterpret_cast<const __nv_bfloat16*>(weight);
  p.dy = reinterpret_cast<const __nv_bfloat16*>(dy);
  p.dh = dh;
  p.dx = dx;
  p.dx16 = reinterpret_cast<__nv_bfloat16*>(dx16);
  p.partial = static_cast<float*>(ws);
  p.rows = rows;
  p.width = width;
  p.eps = eps;
  const int ctas = (int)std::min<int64_t>(rows, kBwdCtas);
  const bool vec = width % 8 == 0 && aligned16({h, weight, dy, dh, dx, dx16});
  TSP_TRY(h_f32 ? launch_bwd_res<RES_F32>(p, vec, ctas, s) : launch_bwd_res<RES_BF16>(p, vec, ctas, s));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "rmsnorm backward: launch");
  rmsnorm_dw_kernel<<<(width + 31) / 32, 1024, 0, s>>>(p.partial, ctas, width, dw);
  e = cudaGetLastError();
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "rmsnorm backward: dw launch");
}

}  // extern "C"
