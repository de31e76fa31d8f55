// attention_math.cuh - the exponential of the attention kernels.
#pragma once

#include "tsp_device.cuh"

namespace tsp {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// P = exp2(s * scale - m) for one row of 128 scores: bf16 pairs stored to TMEM
// (64 columns at p_tmem); returns the row sum. The argument and the sum use packed
// f32x2 FMA/ADD (two elements per instruction): the softmax is bound by instruction
// issue, not by the exponential unit (moving part of the exponentials to an FMA-pipe
// polynomial measured slower).
template <int KT>
__device__ __forceinline__ float exp_tile(const float (&sc)[KT], uint32_t p_tmem, float scale,
                                          float neg_ref) {
  const uint64_t scale2 = f2_pack(scale, scale), nref2 = f2_pack(neg_ref, neg_ref);
  uint64_t sum2[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < KT; c += 16) {
    uint32_t r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(sc[c + 2 * e], sc[c + 2 * e + 1]), scale2, nref2), x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
      r[e] = pack_bf16x2(p0, p1);
    }
    tmem_st8(p_tmem + (uint32_t)(c / 2), r);
  }
  const uint64_t s01 = f2_add(sum2[0], sum2[1]);
  float a, b;
  f2_unpack(s01, a, b);
  return a + b;
}

}  // namespace tsp
