// e4m3.cuh - values of 8 bits (4 exponent and 3 mantissa bits, largest 448) with an fp32 scale for
// each group, as the norm's 8-bit output and the quantiser write them.
#pragma once

#include <cuda_fp8.h>

#include "tsp_device.cuh"

namespace tsp {

constexpr float kE4m3Max = 448.0f;

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

// The same e4m3 values with two operations for two quotients instead of six, for most scales: y (hi + lo), hi + lo
// the reciprocal to 46 bits, rounded once. hi is rounded down, so that lo is not negative and a zero keeps its
// sign.
//
// Before its rounding the result is off by at most 2^-45 of the quotient: lo, which is up to 2^-23 of the
// reciprocal, by 1.5 x 2^-23 of itself, and the product y lo by 2^-24. It can round to the wrong fp32 number only if
// the quotient is that near to a midpoint of two, and that changes the e4m3 value only if one of the two is
// a tie t, halfway between e4m3 values and so of five bits at most. With y = X 2^a and scale = S 2^b, X and S
// of 24 bits, such a midpoint is m 2^c with m a multiple of 2^20, plus or minus 1, and X 2^24 (or 2^25) - m S an
// integer of at most 16: S is then within 16 of a multiple of 2^20. It is not such a multiple itself (the integer would be one
// too, so zero, and a quotient of two numbers of 24 bits is never a midpoint). Scales within 16 of a multiple of
// 2^19, and very small, large or not finite ones, take the other way.
struct QuickQuotient {
  float hi, lo;
  bool ok;
  __device__ __forceinline__ explicit QuickQuotient(float scale) {
    hi = __frcp_rd(scale);
    lo = __fmul_rn(fmaf(-scale, hi, 1.f), hi);
    const uint32_t low = __float_as_uint(scale) & 0x7ffffu;
    ok = scale > 1e-18f && scale < 1e18f && (low == 0u || low - 17u < 0x80000u - 33u);
  }
  __device__ __forceinline__ void pair(float& a, float& b) const {
    const uint64_t y = f2_pack(a, b);
    f2_unpack(f2_fma(y, f2_pack(hi, hi), f2_mul(y, f2_pack(lo, lo))), a, b);
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

}  // namespace tsp
