// rmsnorm.cu - root-mean-square norm with the residual's addition, forward (bf16 or
// e4m3 output) and backward: the step between two blocks of a pre-norm stack.
//
// Forward, per row of `width` elements (sums in fp32):
//     h = x + r            stored in r's type (bf16 or fp32); h = x without a residual
//     y = h * rstd * w,    rstd = 1 / sqrt(mean(h^2) + eps), from the unrounded h
//     e4m3: per row or per 128 columns  scale = max|y| / 448,  y8 = e4m3(y / scale), both
//     quotients in fp32
// Backward, with g = dy * w and n = width:
//     dx = rstd * g - h * rstd^3 * (sum(g h) / n)  (+ dh)
//     dw = sum over rows of dy * h * rstd
// rstd is taken again from h: the row is in registers for sum(g h) in any case, so a
// saved rstd would only add traffic.
//
// Bound: HBM. A row is read once, stays on chip between its reduction and its outputs, and
// is written once. Layout of the work: a row of up to 1024 elements per warp (no block
// barrier), a longer one per CTA; each thread owns the same columns of every row it meets,
// so the weight is loaded once and dw is summed in registers. CTAs are persistent and copy
// their next rows into shared memory (cp.async) while they work on the current one. A
// thread's columns come in pieces of 16 bytes of the widest operand (8 columns of bf16, 4
// of fp32), so that every copy of a warp is contiguous: 8 columns of an fp32 stream per
// thread made each copy fetch half sectors (16384 x 4096: 157 us against 135).
// 16384 x 4096, of the measured copy rate: fp32 stream 128 us (0.93), e4m3 beside a bf16
// stream 78 us (0.90), backward 88 us (0.90); backward of an fp32 stream 170 us (0.81), with dx
// over dh and a bf16 copy of dx 184 us (0.86).
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

// VEC consecutive elements as fp32: 8 or 4 (one 16- or 8-byte access of bf16) or 1.
template <int VEC>
__device__ __forceinline__ void load_bf16(const void* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *static_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else if constexpr (VEC == 4) {
    const uint2 u = *static_cast<const uint2*>(p);
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  } else {
    v[0] = __bfloat162float(*static_cast<const __nv_bfloat16*>(p));
  }
}

template <int VEC>
__device__ __forceinline__ void load_f32(const void* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = *static_cast<const float*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 a = static_cast<const float4*>(p)[i];
      v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
    }
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
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

template <int VEC>
__device__ __forceinline__ void store_f32(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
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

// Columns per piece of the staged kernels.
template <int RES>
constexpr int piece_of = RES == RES_F32 ? 4 : 8;

// A piece of BYTES from global to shared memory, asynchronously.
template <int BYTES>
__device__ __forceinline__ void copy_ahead(void* smem, const void* global) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(global) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(smem)), "l"(global) : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait_all_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// The scale of a group whose largest |y| has the bits `top`: top / 448, rounded to nearest (the
// product with the reciprocal, and its remainder, exact in an fma, times the reciprocal; a
// quotient by 448 = 7 x 64 is never near halfway between two numbers). A group of zeros takes 1;
// the smallest scale is the smallest normal number, so that its reciprocal is finite.
// NaN or infinity in the group gives a NaN or infinite scale.
__device__ __forceinline__ float e4m3_scale(uint32_t top) {
  const float t = __uint_as_float(top);
  if (top == 0u) return 1.f;
  if (top >= 0x7f800000u) return t;
  constexpr float r = 1.f / kE4m3Max;
  const float q = t * r;
  return fmaxf(fmaf(fmaf(-q, kE4m3Max, t), r, q), 1.17549435e-38f);
}

// y / scale, rounded to nearest as the fp32 division is, without a division per element: with
// the correctly rounded reciprocal, each step q - (q scale - y) / scale takes an exact remainder,
// the first leaves less than one unit in the last place and the second none (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990). A product
// with the reciprocal alone is off by a unit, which at a tie between two e4m3 values picks the
// wrong one. Small scales are raised by 2^64, so that the remainders do not underflow. 16384 x 4096
// with groups of 128: 78 us beside a bf16 stream and 120 beside fp32, as without the steps; 66
// instead of 54 without a residual (93, 126 and 75 with the division itself, which the kernel of
// single elements uses: 260 us for 4095 columns beside a bf16 stream, 240 without).
struct Quotient {
  float up, inv, sc;
  __device__ __forceinline__ explicit Quotient(float scale) {
    up = scale < 1e-18f ? 18446744073709551616.f : 1.f;
    inv = __frcp_rn(scale * up);
    sc = isinf(scale) ? 0.f : scale * up;  // no remainders: finite / infinity is 0
  }
  // of two values, in place; from -y, so that a zero keeps its sign
  __device__ __forceinline__ void pair(float& a, float& b) const {
    const uint64_t n = f2_mul(f2_pack(-a, -b), f2_pack(up, up)), ni = f2_pack(-inv, -inv), s = f2_pack(sc, sc);
    uint64_t q = f2_mul(n, ni);
    q = f2_fma(f2_fma(q, s, n), ni, q);
    f2_unpack(f2_fma(f2_fma(q, s, n), ni, q), a, b);
  }
};

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

// One row per CTA straight from global memory, NV times VEC elements per thread: rows of
// single elements (VEC 1), and rows too wide to stage.
template <int VEC, int NV, int RES, bool E4M3>
__global__ void __launch_bounds__(1024) rmsnorm_fwd_kernel(const NormParams p) {
  __shared__ float part[2][32];
  __shared__ uint32_t tops[2][E4M3 ? kMaxWidth / 128 : 32];
  const int tid = threadIdx.x, lanes = blockDim.x;
  const float inv_n = 1.f / (float)p.width;
  float w[NV][VEC], v[NV][VEC];
  auto col = [&](int i) { return (i * lanes + tid) * VEC; };
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < p.width) load_bf16<VEC>(p.w + col(i), w[i]);
  int odd = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, odd ^= 1) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const long long at = row * p.width + col(i);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      if (col(i) < p.width) {
        load_bf16<VEC>(p.x + at, v[i]);
        if constexpr (RES != RES_NONE) {
          float r[VEC];
          load_stream<VEC, RES>(p.r, at, r);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += r[e];
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    const float rstd = 1.f / sqrtf(row_sum<false>(ss, part[odd]) * inv_n + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) >= p.width) continue;
      if constexpr (RES != RES_NONE) store_stream<VEC, RES>(p.h, row * p.width + col(i), v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] *= rstd * w[i][e];
      if constexpr (!E4M3)
        store_bf16<VEC>(static_cast<__nv_bfloat16*>(p.y) + row * p.width + col(i), v[i]);
    }
    if constexpr (E4M3) {
      uint8_t* y8 = static_cast<uint8_t*>(p.y) + row * p.width;
      auto top_of = [&](int i) {
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) t = max(t, __float_as_uint(fabsf(v[i][e])));
        return t;
      };
      auto store8 = [&](int i, float scale) {
        if constexpr (VEC == 8) {
          const Quotient by(scale);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) by.pair(v[i][e], v[i][e + 1]);
        } else {
          v[i][0] = __fdiv_rn(v[i][0], scale);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) y8[col(i) + e] = to_e4m3(v[i][e]);
      };
      if (p.group == 0) {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) t = max(t, top_of(i));
        const float scale = e4m3_scale(row_max<false>(t, tops[odd]));
        if (tid == 0) p.scales[row] = scale;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < p.width) store8(i, scale);
      } else {
        // a warp's columns of one i lie in one group (VEC 1), or a half warp's (VEC 8); the
        // warps of a group meet in shared memory (a maximum does not depend on the order of
        // the atomics)
        const int groups = (p.width + 127) / 128;
        __syncthreads();
        for (int g = threadIdx.x; g < groups; g += blockDim.x) tops[0][g] = 0u;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint32_t t = top_of(i);
#pragma unroll
          for (int o = VEC == 8 ? 8 : 16; o; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
          if (tid % (VEC == 8 ? 16 : 32) == 0 && col(i) < p.width) atomicMax(&tops[0][col(i) / 128], t);
        }
        __syncthreads();
        for (int g = threadIdx.x; g < groups; g += blockDim.x) {
          const float scale = e4m3_scale(tops[0][g]);
          p.scales[row * groups + g] = scale;
          tops[1][g] = __float_as_uint(scale);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < p.width) store8(i, __uint_as_float(tops[1][col(i) / 128]));
      }
    }
  }
}

// Rows staged in shared memory: each thread copies its own pieces of the rows ahead and
// later reads only those, so a wait for its own copies is all the ordering that is needed,
// and STAGES - 1 rows are in flight under the arithmetic and the barriers of the current
// one. One row per warp (WARP) or per CTA.
template <int NV, bool WARP, int RES, bool E4M3, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT, NV * piece_of<RES> > 16 ? 2 : 1024 / MAXT)
    rmsnorm_fwd_staged_kernel(const NormParams p) {
  constexpr int VEC = piece_of<RES>;
  constexpr int XB = 2 * VEC;                       // bytes of a piece of x
  constexpr int RB = RES == RES_NONE ? 0 : 16;      // and of the residual
  extern __shared__ __align__(16) uint8_t ring[];   // [STAGES][NV][threads] pieces of r, then of x
  __shared__ float part[2][32];
  __shared__ uint32_t tops[2][32];
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x, lanes = WARP ? 32 : blockDim.x;
  const long long row0 = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const long long step = WARP ? (long long)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  const float inv_n = 1.f / (float)p.width;
  auto col = [&](int i) { return (i * lanes + tid) * VEC; };
  auto r_at = [&](int stage, int i) { return ring + ((stage * NV + i) * blockDim.x + threadIdx.x) * RB; };
  uint8_t* x_ring = ring + STAGES * NV * blockDim.x * RB;
  auto x_at = [&](int stage, int i) { return x_ring + ((stage * NV + i) * blockDim.x + threadIdx.x) * XB; };
  auto fetch = [&](long long row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) >= p.width) continue;
        const long long at = row * p.width + col(i);
        copy_ahead<XB>(x_at(stage, i), p.x + at);
        if constexpr (RES != RES_NONE)
          copy_ahead<16>(r_at(stage, i), static_cast<const uint8_t*>(p.r) + at * (16 / VEC));
      }
    }
    copies_end_group();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(row0 + s * step, s);
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < p.width) load_bf16<VEC>(p.w + col(i), w[i]);
  int odd = 0, stage = 0;
  for (long long row = row0; row < p.rows; row += step, odd ^= 1) {
    copies_wait_all_but<STAGES - 2>();
    float v[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) < p.width) {
        load_bf16<VEC>(x_at(stage, i), v[i]);
        if constexpr (RES != RES_NONE) {
          float r[VEC];
          load_stream<VEC, RES>(r_at(stage, i), 0, r);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += r[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    // this stage is read; the one before it takes the row furthest ahead
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    const float rstd = 1.f / sqrtf(row_sum<WARP>(ss, part[odd]) * inv_n + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) >= p.width) continue;
      if constexpr (RES != RES_NONE) store_stream<VEC, RES>(p.h, row * p.width + col(i), v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] *= rstd * w[i][e];
      if constexpr (!E4M3)
        store_bf16<VEC>(static_cast<__nv_bfloat16*>(p.y) + row * p.width + col(i), v[i]);
    }
    if constexpr (E4M3) {
      uint8_t* y8 = static_cast<uint8_t*>(p.y) + row * p.width;
      uint32_t top[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        top[i] = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) top[i] = max(top[i], __float_as_uint(fabsf(v[i][e])));
      }
      if (p.group == 0) {
        uint32_t t = top[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) t = max(t, top[i]);
        t = row_max<WARP>(t, tops[odd]);
#pragma unroll
        for (int i = 0; i < NV; ++i) top[i] = t;
        if (tid == 0) p.scales[row] = e4m3_scale(t);
      } else {
        // 128 / VEC consecutive threads hold 128 consecutive columns
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (VEC == 4) {
            top[i] = __reduce_max_sync(0xffffffffu, top[i]);
          } else {
#pragma unroll
            for (int o = 8; o; o >>= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float scale = e4m3_scale(top[i]);
        const Quotient by(scale);
        if (col(i) >= p.width) continue;
        if (p.group != 0 && tid % (128 / VEC) == 0)
          p.scales[row * ((p.width + 127) / 128) + col(i) / 128] = scale;
#pragma unroll
        for (int e = 0; e < VEC; e += 2) by.pair(v[i][e], v[i][e + 1]);
        const uint32_t lo = to_e4m3x4(v[i][0], v[i][1], v[i][2], v[i][3]);
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(y8 + col(i)) = make_uint2(lo, to_e4m3x4(v[i][4], v[i][5], v[i][6], v[i][7]));
        else
          *reinterpret_cast<uint32_t*>(y8 + col(i)) = lo;
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
  int stage_dh;    // dh is staged too (where it fits shared memory)
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
  dependents_may_start();
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

// The same with the rows staged in shared memory, as in the forward: one row per warp (WARP)
// or per CTA. Operands in bf16 stay packed until they are used, so that 1024 threads fit.
template <int NV, bool WARP, int RES, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT, WARP ? 2 : MAXT <= 256 ? 3 : 1)
    rmsnorm_bwd_staged_kernel(const NormBwdParams p) {
  constexpr int VEC = piece_of<RES>;
  constexpr int YB = 2 * VEC;                      // bytes of a piece of dy
  extern __shared__ __align__(16) uint8_t ring[];  // [STAGES][NV][threads] pieces of h, dh, dy
  __shared__ float part[2][2][32];
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x, lanes = WARP ? 32 : blockDim.x;
  const long long row0 = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const long long step = WARP ? (long long)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  const bool has_dh = p.dh != nullptr, stage_dh = p.stage_dh != 0;
  const float inv_n = 1.f / (float)p.width;
  const int each = STAGES * NV * blockDim.x * 16;
  dependents_may_start();
  auto col = [&](int i) { return (i * lanes + tid) * VEC; };
  auto slot = [&](int stage, int i) { return (stage * NV + i) * (int)blockDim.x + (int)threadIdx.x; };
  auto h_at = [&](int stage, int i) { return ring + slot(stage, i) * 16; };
  auto d_at = [&](int stage, int i) { return ring + each + slot(stage, i) * 16; };
  uint8_t* y_ring = ring + (stage_dh ? 2 : 1) * each;
  auto y_at = [&](int stage, int i) { return y_ring + slot(stage, i) * YB; };
  auto fetch = [&](long long row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) >= p.width) continue;
        const long long at = row * p.width + col(i);
        copy_ahead<16>(h_at(stage, i), static_cast<const uint8_t*>(p.h) + at * (16 / VEC));
        if (stage_dh) copy_ahead<16>(d_at(stage, i), static_cast<const uint8_t*>(p.dh) + at * (16 / VEC));
        copy_ahead<YB>(y_at(stage, i), p.dy + at);
      }
    }
    copies_end_group();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(row0 + s * step, s);
  uint32_t w[NV][VEC / 2], g[NV][VEC / 2];  // bf16 pairs
  float dw[NV][VEC];
  auto pieces = [](const void* from, uint32_t (&to)[VEC / 2]) {
    if constexpr (VEC == 8) {
      const uint4 u = *static_cast<const uint4*>(from);
      to[0] = u.x, to[1] = u.y, to[2] = u.z, to[3] = u.w;
    } else {
      const uint2 u = *static_cast<const uint2*>(from);
      to[0] = u.x, to[1] = u.y;
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) w[i][e] = g[i][e] = 0u;
    if (col(i) < p.width) pieces(p.w + col(i), w[i]);
  }
  int odd = 0, stage = 0;
  for (long long row = row0; row < p.rows; row += step, odd ^= 1) {
    copies_wait_all_but<STAGES - 2>();
    float h[NV][VEC];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[i][e] = 0.f;
      if (col(i) < p.width) {
        load_stream<VEC, RES>(h_at(stage, i), 0, h[i]);
        pieces(y_at(stage, i), g[i]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float wy = e & 1 ? bf16_hi(g[i][e / 2]) * bf16_hi(w[i][e / 2])
                               : bf16_lo(g[i][e / 2]) * bf16_lo(w[i][e / 2]);
        ss = fmaf(h[i][e], h[i][e], ss);
        sg = fmaf(wy, h[i][e], sg);
      }
    }
    // the stage of the row before is read to its end: the row furthest ahead goes there
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    // both sums behind one barrier
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    if constexpr (!WARP) {
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
    }
    const float rstd = 1.f / sqrtf(ss * inv_n + p.eps);
    const float coef = rstd * rstd * (sg * inv_n);  // dx = rstd (g - h coef)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (c >= p.width) continue;
      float d[VEC];
      if (stage_dh) load_stream<VEC, RES>(d_at(stage, i), 0, d);
      else if (has_dh) load_stream<VEC, RES>(p.dh, row * p.width + c, d);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float y = e & 1 ? bf16_hi(g[i][e / 2]) : bf16_lo(g[i][e / 2]);
        const float wt = e & 1 ? bf16_hi(w[i][e / 2]) : bf16_lo(w[i][e / 2]);
        const float t = rstd * (y * wt - h[i][e] * coef);
        dw[i][e] = fmaf(y, h[i][e] * rstd, dw[i][e]);
        d[e] = has_dh ? d[e] + t : t;
      }
      store_stream<VEC, RES>(p.dx, row * p.width + c, d);
      if (p.dx16 != nullptr) store_bf16<VEC>(p.dx16 + row * p.width + c, d);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  float* out = p.partial + (long long)blockIdx.x * p.width;
  if constexpr (WARP) {
    // the warps' sums one after the other, in the ring's memory (every warp is done with it)
    float* sum = reinterpret_cast<float*>(ring);
    copies_wait_all_but<0>();
    __syncthreads();
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k) {
      if ((int)(threadIdx.x >> 5) == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (col(i) >= p.width) continue;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (k > 0) dw[i][e] += sum[col(i) + e];
            sum[col(i) + e] = dw[i][e];
          }
          if (k == (int)(blockDim.x >> 5) - 1) store_f32<VEC>(out + col(i), dw[i]);
        }
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col(i) < p.width) store_f32<VEC>(out + col(i), dw[i]);
  }
}

// Rows that are not made of whole pieces (odd widths, unaligned buffers). The backward copies
// the aligned 16-byte spans that cover a row, one row ahead, and works on single elements of
// the copy. A span's bytes outside the row are ignored; spans that leave the buffer are
// copied element by element. (16384 x 4095: 228 us, 430 without copies. The forward, with fewer
// operands, is faster without.)
template <class E>
__device__ __forceinline__ const E* copy_row(uint8_t* smem, const E* buffer, long long row, long long rows,
                                             int width) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(buffer);
  const uintptr_t hi = lo + (uintptr_t)rows * (uintptr_t)width * sizeof(E);
  const uintptr_t at = lo + (uintptr_t)row * (uintptr_t)width * sizeof(E);
  const uintptr_t first = at & ~(uintptr_t)15;
  if (row < rows) {
    const int spans = (int)((at - first + (uintptr_t)width * sizeof(E) + 15) >> 4);
    for (int k = threadIdx.x; k < spans; k += blockDim.x) {
      const uintptr_t src = first + 16u * (unsigned)k;
      if (src >= lo && src + 16 <= hi) {
        copy_ahead<16>(smem + 16 * k, reinterpret_cast<const void*>(src));
      } else {
#pragma unroll
        for (unsigned e = 0; e < 16; e += sizeof(E))
          if (src + e >= lo && src + e < hi)
            *reinterpret_cast<E*>(smem + 16 * k + e) = *reinterpret_cast<const E*>(src + e);
      }
    }
  }
  return reinterpret_cast<const E*>(smem + (at - first));
}
// Shared memory of a copied row of `width` elements.
__host__ __device__ constexpr int row_bytes(int width, int element) {
  return (width * element + 15 + 15) / 16 * 16;
}
template <int RES>
struct StreamOf {
  using type = __nv_bfloat16;
};
template <>
struct StreamOf<RES_F32> {
  using type = float;
};
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// dw is summed in shared memory, each column by the thread that owns it.
template <int RES>
__global__ void __launch_bounds__(512, 2) rmsnorm_bwd_odd_kernel(const NormBwdParams p) {
  using R = typename StreamOf<RES>::type;
  extern __shared__ __align__(16) uint8_t ring[];  // dw, then two copies of h, dy (and dh)
  __shared__ float part[2][2][32];
  float* dw = reinterpret_cast<float*>(ring);
  const bool has_dh = p.dh != nullptr;
  const int hb = row_bytes(p.width, sizeof(R)), yb = row_bytes(p.width, 2);
  const int tid = threadIdx.x, threads = blockDim.x;
  const float inv_n = 1.f / (float)p.width;
  dependents_may_start();
  struct Row {
    const R* h;
    const R* d;
    const __nv_bfloat16* y;
  };
  auto fetch = [&](long long row, int stage) {
    uint8_t* to = ring + row_bytes(p.width, 4) + stage * (hb + yb + (has_dh ? hb : 0));
    Row r;
    r.h = copy_row(to, static_cast<const R*>(p.h), row, p.rows, p.width);
    r.y = copy_row(to + hb, p.dy, row, p.rows, p.width);
    r.d = has_dh ? copy_row(to + hb + yb, static_cast<const R*>(p.dh), row, p.rows, p.width) : nullptr;
    copies_end_group();
    return r;
  };
  for (int c = tid; c < p.width; c += threads) dw[c] = 0.f;
  Row now = fetch(blockIdx.x, 0);
  int odd = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, odd ^= 1) {
    const Row next = fetch(row + gridDim.x, odd ^ 1);
    copies_wait_all_but<1>();
    __syncthreads();
    float ss = 0.f, sg = 0.f;
#pragma unroll 4
    for (int c = tid; c < p.width; c += threads) {
      const float h = as_float(now.h[c]);
      ss = fmaf(h, h, ss);
      sg = fmaf(__bfloat162float(now.y[c]) * __bfloat162float(p.w[c]), h, sg);
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
    const bool in = (tid & 31) < (threads >> 5);
    ss = in ? part[odd][0][tid & 31] : 0.f;
    sg = in ? part[odd][1][tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    const float rstd = 1.f / sqrtf(ss * inv_n + p.eps);
    const float coef = rstd * rstd * (sg * inv_n);  // dx = rstd (g - h coef)
    R* dx = static_cast<R*>(p.dx) + row * p.width;
    __nv_bfloat16* dx16 = p.dx16 == nullptr ? nullptr : p.dx16 + row * p.width;
#pragma unroll 4
    for (int c = tid; c < p.width; c += threads) {
      const float h = as_float(now.h[c]), y = __bfloat162float(now.y[c]);
      float t = rstd * (y * __bfloat162float(p.w[c]) - h * coef);
      dw[c] = fmaf(y, h * rstd, dw[c]);
      if (has_dh) t += as_float(now.d[c]);
      store_as(dx + c, t);
      if (dx16 != nullptr) dx16[c] = __float2bfloat16_rn(t);
    }
    __syncthreads();  // the copies are read: the row after the next goes there
    now = next;
  }
  for (int c = tid; c < p.width; c += threads) p.partial[(long long)blockIdx.x * p.width + c] = dw[c];
}

// dw[c] = sum of the partial rows, in a fixed order: 32 row groups per column, then their
// sum.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* partial, int n, int width, float* dw) {
  __shared__ float part[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.f;
  prior_kernel_done();
  if (c < width)
    for (int r = ry; r < n; r += 32) s += __ldcg(partial + (long long)r * width + c);
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

// Threads of a CTA that holds a row of `items` (pieces or elements), nv per thread.
int row_threads(int items, int nv) { return ((items + nv - 1) / nv + 31) / 32 * 32; }

// Threads of a CTA on a row of single elements: about eight columns each.
int odd_threads(int width) { return width <= 1024 ? 128 : width <= 2048 ? 256 : 512; }

template <int VEC, int NV, int RES, bool E4M3>
tsp_status launch_fwd_direct(const NormParams& p, cudaStream_t s) {
  const int threads = row_threads((p.width + VEC - 1) / VEC, NV);
  const long long cap = (long long)sm_count() * std::max(1, 1024 / threads);
  rmsnorm_fwd_kernel<VEC, NV, RES, E4M3><<<(unsigned)std::min<long long>(p.rows, cap), threads, 0, s>>>(p);
  return TSP_OK;
}

template <int NV, bool WARP, int RES, bool E4M3, int STAGES, int MAXT>
tsp_status launch_fwd_staged(const NormParams& p, int threads, cudaStream_t s) {
  auto kernel = rmsnorm_fwd_staged_kernel<NV, WARP, RES, E4M3, STAGES, MAXT>;
  const size_t smem = (size_t)STAGES * NV * threads * (2 * piece_of<RES> + (RES == RES_NONE ? 0 : 16));
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                            "rmsnorm: cudaFuncSetAttribute"));
  // resident CTAs: by registers (1024 threads, half of them with 32 columns each) and by
  // shared memory
  const int by_regs = NV * piece_of<RES> > 16 ? 2 : std::max(1, 1024 / threads);
  const long long per_sm = std::min<long long>(by_regs, (220 * 1024) / (long long)smem);
  const long long cap = (long long)sm_count() * std::max<long long>(1, per_sm);
  const long long blocks = WARP ? (p.rows + threads / 32 - 1) / (threads / 32) : p.rows;
  kernel<<<(unsigned)std::min(blocks, cap), threads, smem, s>>>(p);
  return TSP_OK;
}

// vec: rows are whole pieces. A warp takes a row of up to 32 columns per lane; a CTA 16 per
// thread. The fewer bytes a warp has per row, the more rows are staged ahead.
template <int RES, bool E4M3>
tsp_status launch_fwd_res(const NormParams& p, bool vec, cudaStream_t s) {
  constexpr int P = 8 / piece_of<RES>;  // pieces per 8 columns
  if (!vec) {
    if (p.width <= 4096) return launch_fwd_direct<1, 8, RES, E4M3>(p, s);
    return launch_fwd_direct<1, 32, RES, E4M3>(p, s);
  }
  if (p.width <= 256) return launch_fwd_staged<P, true, RES, E4M3, 4, 256>(p, 256, s);
  if (p.width <= 512) return launch_fwd_staged<2 * P, true, RES, E4M3, 3, 256>(p, 256, s);
  if (p.width <= 1024) return launch_fwd_staged<4 * P, true, RES, E4M3, 2, 256>(p, 256, s);
  const int threads = row_threads(p.width / 8, 2);
  // an fp32 stream beside a bf16 output moves the most bytes per column: with at least four CTAs to
  // a multiprocessor, their loads in flight keep up without staging (67M elements, direct against
  // staged: 138 us against 143 at 1032 columns, 123 against 135 at 2048, 128 against 135 at 4096;
  // with fewer CTAs 136 and 136 at 4608 and 8192, 132 against 136 at 5120, but 147 against 136 at
  // 6144 and 175 against 136 at 12288). Every other kind gains from staging (e4m3 beside bf16 at
  // 4096: 78 us against 97).
  if (threads <= 256) {
    if constexpr (RES == RES_F32 && !E4M3) return launch_fwd_direct<8, 2, RES, E4M3>(p, s);
    else return launch_fwd_staged<2 * P, false, RES, E4M3, 2, 256>(p, threads, s);
  }
  if (threads <= 1024) return launch_fwd_staged<2 * P, false, RES, E4M3, 2, 1024>(p, threads, s);
  return launch_fwd_direct<8, 4, RES, E4M3>(p, s);
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
tsp_status launch_bwd_direct(const NormBwdParams& p, int ctas, cudaStream_t s) {
  rmsnorm_bwd_kernel<VEC, NV, RES>
      <<<ctas, row_threads((p.width + VEC - 1) / VEC, NV), 0, s>>>(p);
  return TSP_OK;
}

template <int NV, bool WARP, int RES, int STAGES, int MAXT>
tsp_status launch_bwd_staged(NormBwdParams p, int ctas, int threads, cudaStream_t s) {
  auto kernel = rmsnorm_bwd_staged_kernel<NV, WARP, RES, STAGES, MAXT>;
  const size_t piece = (size_t)STAGES * NV * threads;
  const size_t lean = piece * (2 * piece_of<RES> + 16), most = lean + piece * 16;
  p.stage_dh = p.dh != nullptr && most <= 220 * 1024;
  const size_t smem = p.stage_dh ? most : lean;
  TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                            "rmsnorm backward: cudaFuncSetAttribute"));
  kernel<<<ctas, threads, smem, s>>>(p);
  return TSP_OK;
}

// How the backward covers a row of whole pieces, and with how many CTAs (those that fit the
// GPU at a time: three per SM of up to 256 threads, two where a warp takes a row, one of
// more threads).
int bwd_ctas(int64_t rows, int width, bool vec) {
  const int threads = row_threads(width / 8, 2);
  const int most = !vec ? kBwdCtas : width <= 1024 ? kBwdCtas / 3 * 2 : threads <= 256 ? kBwdCtas : kBwdCtas / 3;
  return (int)std::min<int64_t>(rows, most);
}

template <int RES>
tsp_status launch_bwd_res(const NormBwdParams& p, bool vec, int ctas, cudaStream_t s) {
  constexpr int P = 8 / piece_of<RES>;
  if (!vec) {
    const int hb = row_bytes(p.width, RES == RES_F32 ? 4 : 2);
    const size_t smem = row_bytes(p.width, 4) + 2 * (row_bytes(p.width, 2) + (p.dh ? 2 : 1) * hb);
    if (smem > 220 * 1024) return launch_bwd_direct<1, 32, RES>(p, ctas, s);
    auto kernel = rmsnorm_bwd_odd_kernel<RES>;
    TSP_TRY(ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem,
                              "rmsnorm backward: cudaFuncSetAttribute"));
    kernel<<<ctas, odd_threads(p.width), smem, s>>>(p);
    return TSP_OK;
  }
  if (p.width <= 256) return launch_bwd_staged<P, true, RES, 4, 256>(p, ctas, 256, s);
  if (p.width <= 512) return launch_bwd_staged<2 * P, true, RES, 3, 256>(p, ctas, 256, s);
  if (p.width <= 1024) return launch_bwd_staged<4 * P, true, RES, 2, 256>(p, ctas, 256, s);
  const int threads = row_threads(p.width / 8, 2);
  if (threads <= 128) return launch_bwd_staged<2 * P, false, RES, 4, 128>(p, ctas, threads, s);
  if (threads <= 256) return launch_bwd_staged<2 * P, false, RES, 2, 256>(p, ctas, threads, s);
  if (threads <= 512) return launch_bwd_staged<2 * P, false, RES, P == 1 ? 3 : 2, 512>(p, ctas, threads, s);
  if (threads <= 1024) return launch_bwd_staged<2 * P, false, RES, 2, 1024>(p, ctas, threads, s);
  return launch_bwd_direct<8, 4, RES>(p, ctas, s);
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
  TSP_GUARD_BEGIN
  return rmsnorm_fwd("tsp_rmsnorm_fwd", rows, width, x, residual, residual_f32, weight, eps, h, y,
                     false, 0, nullptr, static_cast<cudaStream_t>(stream));
  TSP_GUARD_END
}

tsp_status tsp_rmsnorm_fwd_e4m3(int64_t rows, int width, const tsp_bf16* x, const void* residual,
                                int residual_f32, const tsp_bf16* weight, float eps, int group,
                                void* h, uint8_t* y, float* scales, void* stream) {
  TSP_GUARD_BEGIN
  if (group != 0 && group != 128)
    return fail(TSP_ERR_UNSUPPORTED, "tsp_rmsnorm_fwd_e4m3: group 0 (a row) or 128 columns");
  return rmsnorm_fwd("tsp_rmsnorm_fwd_e4m3", rows, width, x, residual, residual_f32, weight, eps, h,
                     y, true, group, scales, static_cast<cudaStream_t>(stream));
  TSP_GUARD_END
}

size_t tsp_rmsnorm_workspace_bytes(int64_t rows, int width) {
  if (rows < 0 || width < 1 || width > kMaxWidth) return 0;
  const int64_t ctas = rows < kBwdCtas ? (rows < 1 ? 1 : rows) : kBwdCtas;
  return align256((size_t)ctas * (size_t)width * sizeof(float));
}

tsp_status tsp_rmsnorm_bwd(int64_t rows, int width, const void* h, int h_f32, const tsp_bf16* weight,
                           float eps, const tsp_bf16* dy, const void* dh, void* dx, tsp_bf16* dx16,
                           float* dw, void* ws, void* stream) {
  TSP_GUARD_BEGIN
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
  const bool vec = width % 8 == 0 && aligned16({h, weight, dy, dh, dx, dx16});
  const int ctas = bwd_ctas(rows, width, vec);
  TSP_TRY(h_f32 ? launch_bwd_res<RES_F32>(p, vec, ctas, s) : launch_bwd_res<RES_BF16>(p, vec, ctas, s));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "rmsnorm backward: launch");
  e = launch_early(rmsnorm_dw_kernel, (width + 31) / 32, 1024, 0, s, p.partial, ctas, width, dw);
  return e == cudaSuccess ? TSP_OK : cuda_fail(e, "rmsnorm backward: dw launch");
  TSP_GUARD_END
}

}  // extern "C"
