// adamw.cu - one AdamW step over a list of tensors:
//     g' = g min(1, max_norm / (norm + 1e-6))      with a norm given, g otherwise
//     m  = beta1 m + (1 - beta1) g'                 v = beta2 v + (1 - beta2) g'^2
//     p  = p - lr (decay p + (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps))
// Weights are fp32, bf16, or bf16 beside an fp32 master that holds them exactly; m and v are fp32,
// or e4m3 with an fp32 scale for each 128 elements of a tensor.
//
// Bound: HBM. Every value is read once and written once, clipping included (the factor is formed
// from the norm here, so the gradients are not scaled in a pass of their own). 202M bf16 weights with fp32
// masters: 866 us with 32-bit states (7.0 TB/s), 632 to 637 with 8-bit ones (5.8 TB/s; 100 instructions an element,
// 0.8 per cycle and scheduler, bind as much); fp32 weights 803 and 600. bf16 weights without masters are the one form
// that 8 bits make slower, 640 and 684 (3.0 TB/s): each element takes a second hash. As in grad_clip.cu
// the list travels in the kernels' parameters, cut into chunks of a CTA each (persistent CTAs that take
// them in turn: 202M weights with masters 941 us, one CTA each 866). A tensor without a gradient between two others
// ends a launch.
//
// Roundings. All arithmetic is fp32 on the values that the states stand for. 8-bit states are
// rounded stochastically, up with the probability of the distance from the lower neighbour: one
// step moves v by about 1 - beta2 of itself, far below half of an e4m3 step, so rounding to nearest
// would freeze it. A v above zero is never rounded to zero, which would make the step m / eps. A bf16
// weight without a master is rounded stochastically too, for the same reason. The random bits are a
// hash of seed, step, tensor and element, so that a step is reproducible.
#include <algorithm>
#include <cmath>
#include <vector>

#include "e4m3.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace {

constexpr int kChunk = 4096;
constexpr int kThreads = 256;
constexpr int kSmall = 64;   // tensors per launch in the small table (4.5 KB of parameters)
constexpr int kLarge = 400;  // and in the large one

enum : unsigned char { GRAD_BF16 = 1, PARAM_BF16 = 2, MASTER = 4, ALIGNED = 8 };

template <int N>
struct Table {
  void* p[N];    // the weight, or its master
  void* p16[N];  // MASTER: the bf16 weight
  const void* g[N];
  void* m[N];
  void* v[N];
  float* ms[N];
  float* vs[N];
  unsigned long long n[N];    // elements
  unsigned int first[N + 1];  // first chunk
  unsigned char kind[N];
  int count;
  int index0;  // place of the first tensor in the call's list
};

struct Step {
  float beta1, beta2, one_beta1, one_beta2, eps;
  float rate, root, shrink;  // of Shared, where neither lr nor t is on the device
  float max_norm;
  double lr, decay, log_beta1, log_beta2;
  long long t;
  unsigned int seed;
  const float* norm;
  const float* device_lr;
  const long long* device_t;
};

// What every element of a step shares.
struct Shared {
  float factor;        // of the gradient
  float rate, root;    // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float shrink;        // lr decay
  unsigned int key;    // of the random bits
};

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7A35E9B5u;
  x = (x ^ (x >> 15)) * 0x68E31DA5u;
  return x ^ (x >> 16);
}

// 32 random bits for an element; high: of the upper half of its number, the same for all of a chunk.
__device__ __forceinline__ uint32_t random_bits(uint32_t key, uint32_t element, uint32_t high) {
  return mix((element ^ key) + high);
}
__device__ __forceinline__ uint32_t high_bits(unsigned long long chunk_at) { return (uint32_t)(chunk_at >> 32) * 0x9E3779B1u; }

__device__ __forceinline__ void make_shared(const Step& a, Shared& s) {
  const long long t = a.device_t ? *a.device_t : a.t;
  s.rate = a.rate, s.root = a.root, s.shrink = a.shrink;
  if (a.device_t || a.device_lr) {
    const double lr = a.device_lr ? (double)*a.device_lr : a.lr;
    s.rate = (float)(lr / -expm1((double)t * a.log_beta1));
    s.root = (float)(1. / sqrt(-expm1((double)t * a.log_beta2)));
    s.shrink = (float)(lr * a.decay);
  }
  s.key = mix(a.seed + (unsigned int)t);
  s.factor = 1.f;
  if (a.norm) {
    // an infinite max_norm clips nothing, not even an infinite norm; a NaN norm stays one
    const float v = *a.norm;
    const float want = isinf(a.max_norm) && !isnan(v) ? 1.f : __fdiv_rn(a.max_norm, __fadd_rn(v, 1e-6f));
    s.factor = want >= 1.f ? 1.f : want;
  }
}

// The byte `b` of each of four words.
__device__ __forceinline__ uint32_t bytes_of(const uint32_t (&x)[4], int b) {
  return __byte_perm(__byte_perm(x[0], x[1], b | ((4 + b) << 4)), __byte_perm(x[2], x[3], b | ((4 + b) << 4)), 0x5410);
}

// The e4m3 codes of four quotients x * inv, |x * inv| <= 448 but for its rounding, each rounded to a neighbouring
// value: 16 random bits of the 20 that a value lacks are added before they are cut off. Below 2^-6 the
// values are 2^-9 apart: floor(512 |q| + u), the floor by an addition that rounds down. Conversions between
// integers and floating point, and roundings by instructions of their own, run at a fourth of this
// arithmetic's rate or less. SQUARES: x is not negative, small quotients are common (not looked for), and
// what is above zero stays so.
template <bool SQUARES>
__device__ __forceinline__ uint32_t stochastic8(const float (&x)[4], float inv, const uint32_t (&r16)[4]) {
  uint32_t code[4], q[4];  // the code in the third byte
  uint32_t least = 0xffffffffu;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float product = x[e] * inv;
    q[e] = __float_as_uint(fminf(SQUARES ? product : fabsf(product), kE4m3Max));
    code[e] = (q[e] >> 4) + r16[e] - (120u << 19);
    least = min(least, q[e]);
  }
  if (SQUARES || least < 0x3c800000u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = __uint_as_float(0x3f800000u | (r16[e] << 7)) - 1.f;  // r16 / 65536
      uint32_t c = __float_as_uint(__fadd_rd(fmaf(__uint_as_float(q[e]), 512.f, u), 8388608.f)) & 15u;
      if (SQUARES) c = max(c, min(__float_as_uint(x[e]), 1u));
      if (q[e] < 0x3c800000u) code[e] = c << 16;
    }
  }
  const uint32_t codes = bytes_of(code, 2);
  if (SQUARES) return codes;
  const uint32_t bits[4] = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  return codes | (bytes_of(bits, 3) & 0x80808080u);
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(__half2(h));
}

// Four elements of a tensor per thread: consecutive ones where everything is aligned (VEC), else a
// warp's width apart. FULL: all of them exist.
template <bool VEC, bool FULL>
struct Four {
  unsigned long long at;  // the first
  int left;               // elements from it to the end of the chunk (FULL: enough)
  __device__ __forceinline__ bool has(int e) const { return FULL || (VEC ? e : 32 * e) < left; }
  __device__ __forceinline__ unsigned long long of(int e) const { return at + (VEC ? e : 32 * e); }

  __device__ __forceinline__ void load32(const void* p, float (&x)[4]) const {
    const float* f = static_cast<const float*>(p);
    if (VEC && has(3)) {
      const float4 u = *reinterpret_cast<const float4*>(f + at);
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = has(e) ? f[of(e)] : 0.f;
    }
  }
  __device__ __forceinline__ void load16(const void* p, float (&x)[4]) const {
    const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(p);
    if (VEC && has(3)) {
      const uint2 u = *reinterpret_cast<const uint2*>(f + at);
      x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = has(e) ? __bfloat162float(f[of(e)]) : 0.f;
    }
  }
  __device__ __forceinline__ void load8(const void* p, float scale, float (&x)[4]) const {
    const uint8_t* f = static_cast<const uint8_t*>(p);
    uint32_t u = 0;
    if (VEC && has(3)) {
      u = *reinterpret_cast<const uint32_t*>(f + at);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (has(e)) u |= (uint32_t)f[of(e)] << (8 * e);
    }
    const float2 lo = from_e4m3x2(u & 0xffffu), hi = from_e4m3x2(u >> 16);
    x[0] = lo.x * scale, x[1] = lo.y * scale, x[2] = hi.x * scale, x[3] = hi.y * scale;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!has(e)) x[e] = 0.f;  // whatever the scale
  }
  __device__ __forceinline__ void store32(void* p, const float (&x)[4]) const {
    float* f = static_cast<float*>(p);
    if (VEC && has(3)) {
      *reinterpret_cast<float4*>(f + at) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (has(e)) f[of(e)] = x[e];
    }
  }
  __device__ __forceinline__ void store16(void* p, const float (&x)[4]) const {
    __nv_bfloat16* f = static_cast<__nv_bfloat16*>(p);
    if (VEC && has(3)) {
      *reinterpret_cast<uint2*>(f + at) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (has(e)) f[of(e)] = __float2bfloat16_rn(x[e]);
    }
  }
  __device__ __forceinline__ void store8(void* p, uint32_t u) const {
    uint8_t* f = static_cast<uint8_t*>(p);
    if (VEC && has(3)) {
      *reinterpret_cast<uint32_t*>(f + at) = u;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (has(e)) f[of(e)] = (uint8_t)(u >> (8 * e));
    }
  }
};

__device__ __forceinline__ uint32_t largest(const float (&x)[4]) {
  uint32_t top = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(fabsf(x[e])));
  return top;
}

// The scale of a block of a state: NaN where one of its values is infinite or NaN. An infinite scale would leave those
// that are above zero infinite, and their weights standing still.
__device__ __forceinline__ float state_scale(uint32_t top) {
  return top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : e4m3_scale(top);
}

// m, v and p from the gradient g. Every product of m and v is rounded by itself: a state's bits follow from
// the formula alone, and with them the border at which its 8 bits are rounded up. The update takes an
// approximate root and quotient, off by two units each. FULL_RANGE: they take numbers below 2^-126 as they are.
// Without, such a v counts as 0 in the root (it would be under 2^-63), and so does such a numerator: see
// tsp_adamw_step for where that is done.
template <bool FULL_RANGE>
__device__ __forceinline__ void update(const Step& a, const Shared& s, float (&p)[4], const float (&g)[4], float (&m)[4],
                                       float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = __fmul_rn(g[e], s.factor);
    m[e] = __fadd_rn(__fmul_rn(a.beta1, m[e]), __fmul_rn(a.one_beta1, x));
    v[e] = __fadd_rn(__fmul_rn(a.beta2, v[e]), __fmul_rn(a.one_beta2, __fmul_rn(x, x)));
    float root, quotient;
    if constexpr (FULL_RANGE) asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v[e]));
    else asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(v[e]));
    const float above = s.rate * m[e], below = fmaf(root, s.root, a.eps);
    if constexpr (FULL_RANGE) asm("div.approx.f32 %0, %1, %2;" : "=f"(quotient) : "f"(above), "f"(below));
    else asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(quotient) : "f"(above), "f"(below));
    p[e] -= fmaf(s.shrink, p[e], quotient);
  }
}

template <int N, class F>
__device__ __forceinline__ void load_weight(const Table<N>& t, int i, const F& f, float (&p)[4], float (&g)[4]) {
  if (t.kind[i] & PARAM_BF16) f.load16(t.p[i], p);
  else f.load32(t.p[i], p);
  if (t.kind[i] & GRAD_BF16) f.load16(t.g[i], g);
  else f.load32(t.g[i], g);
}

template <int N, class F>
__device__ __forceinline__ void store_weight(const Table<N>& t, int i, const F& f, uint32_t key, uint32_t high,
                                             float (&p)[4]) {
  if (t.kind[i] & PARAM_BF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t r = random_bits(key, (uint32_t)f.of(e), high), u = __float_as_uint(p[e]);
      if ((u & 0x7f800000u) != 0x7f800000u) p[e] = __uint_as_float((u + (r & 0xffffu)) & 0xffff0000u);
    }
    f.store16(t.p[i], p);
  } else {
    f.store32(t.p[i], p);
    if (t.kind[i] & MASTER) f.store16(t.p16[i], p);
  }
}

// A chunk, 128 elements per warp and pass. FULL: it is whole. scales: of the chunk's m and v, old ones in, new
// ones out.
template <int N, bool STATE8, bool FULL_RANGE, bool VEC, bool FULL>
__device__ __forceinline__ void update_chunk(const Table<N>& t, int i, unsigned long long chunk_at, int n,
                                             const Step& a, const Shared& s, float (*scales)[kChunk / 128]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tensor_key = mix(s.key + (unsigned int)(t.index0 + i));
  const uint32_t state_key = mix(tensor_key), weight_key = mix(tensor_key + 1u), high = high_bits(chunk_at);
#pragma unroll 1
  for (int pass = 0; pass < kChunk / (4 * kThreads); ++pass) {
    const int b = warp * 128 + pass * 4 * kThreads;
    if (!FULL && b >= n) break;
    const int first = b + (VEC ? 4 * lane : lane);
    const Four<VEC, FULL> f{chunk_at + first, n - first};
    const int block = b >> 7;
    float p[4], g[4], m[4], v[4];
    load_weight(t, i, f, p, g);
    if constexpr (STATE8) {
      f.load8(t.m[i], scales[0][block], m);
      f.load8(t.v[i], scales[1][block], v);
    } else {
      f.load32(t.m[i], m);
      f.load32(t.v[i], v);
    }
    update<FULL_RANGE>(a, s, p, g, m, v);
    store_weight(t, i, f, weight_key, high, p);
    if constexpr (STATE8) {
      const float m_scale = state_scale(__reduce_max_sync(0xffffffffu, largest(m)));
      const float v_scale = state_scale(__reduce_max_sync(0xffffffffu, largest(v)));
      uint32_t low[4], up[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t r = random_bits(state_key, (uint32_t)f.of(e), high);
        low[e] = r & 0xffffu;
        up[e] = r >> 16;
      }
      f.store8(t.m[i], stochastic8<false>(m, __frcp_rn(m_scale), low));
      f.store8(t.v[i], stochastic8<true>(v, __frcp_rn(v_scale), up));
      if (lane == 0) {  // read above by this warp alone
        scales[0][block] = m_scale;
        scales[1][block] = v_scale;
      }
    } else {
      f.store32(t.m[i], m);
      f.store32(t.v[i], v);
    }
  }
}

// Six CTAs per SM: with 56 registers and four of them 8-bit states take 646 us instead of 632.
template <int N, bool STATE8, bool FULL_RANGE>
__global__ void __launch_bounds__(kThreads, 6) adamw_kernel(const __grid_constant__ Table<N> t,
                                                         const __grid_constant__ Step a) {
  __shared__ Shared shared;
  if (threadIdx.x == 0) make_shared(a, shared);
  __syncthreads();
  const Shared s = shared;
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {  // the last tensor whose first chunk is not behind this one
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const unsigned long long at = (unsigned long long)(blockIdx.x - t.first[lo]) * kChunk;
  const int n = (int)min((unsigned long long)kChunk, t.n[lo] - at);
  // The chunk's scales are read and written by one warp each, a line at a time. Where each warp read and wrote its
  // blocks' own, lines were read while their neighbours' values were on their way to them, and a step of
  // 202M weights with masters took 860 us instead of 632.
  __shared__ float scales[2][kChunk / 128];
  float* scale = nullptr;
  if constexpr (STATE8) {
    const int w = threadIdx.x >> 5, block = threadIdx.x & 31;
    static_assert(kChunk / 128 == 32, "a lane for each block");
    if (w < 2 && block * 128 < n) {
      scale = (w ? t.vs : t.ms)[lo] + (at >> 7) + block;
      scales[w][block] = *scale;
    }
    __syncthreads();
  }
  if (!(t.kind[lo] & ALIGNED)) update_chunk<N, STATE8, FULL_RANGE, false, false>(t, lo, at, n, a, s, scales);
  else if (n == kChunk) update_chunk<N, STATE8, FULL_RANGE, true, true>(t, lo, at, n, a, s, scales);
  else update_chunk<N, STATE8, FULL_RANGE, true, false>(t, lo, at, n, a, s, scales);
  if constexpr (STATE8) {
    __syncthreads();
    if (scale) *scale = scales[threadIdx.x >> 5][threadIdx.x & 31];
  }
}

struct List {
  int n;
  void* const* params;
  const int* types;
  void* const* masters;
  const void* const* grads;
  const int* grad_types;
  void* const* m;
  void* const* v;
  float* const* ms;
  float* const* vs;
  const int64_t* sizes;
  int bits;
  bool skipped(int i) const { return sizes[i] == 0 || !grads[i]; }
  void* master(int i) const { return masters ? masters[i] : nullptr; }
};

tsp_status check_list(const char* what, const List& l) {
  const std::string w(what);
  if (l.n < 0 || l.n > TSP_GRAD_MAX_TENSORS) return fail(TSP_ERR_UNSUPPORTED, w + ": 0 to 65536 tensors");
  if (l.bits != 32 && l.bits != 8) return fail(TSP_ERR_UNSUPPORTED, w + ": states of 32 or 8 bits");
  if (l.n == 0) return TSP_OK;
  if (!l.params || !l.types || !l.grads || !l.grad_types || !l.m || !l.v || !l.sizes || (l.bits == 8 && (!l.ms || !l.vs)))
    return fail(TSP_ERR_INVALID_ARG, w + ": null list");
  int64_t total = 0;
  for (int i = 0; i < l.n; ++i) {
    if (l.sizes[i] < 0 || l.sizes[i] > (1ll << 40)) return fail(TSP_ERR_INVALID_ARG, w + ": tensor size out of range");
    if (l.skipped(i)) continue;
    total += (l.sizes[i] + kChunk - 1) / kChunk;
    const int types[2] = {l.types[i], l.grad_types[i]};
    for (int t : types)
      if (t != TSP_F32 && t != TSP_BF16) return fail(TSP_ERR_UNSUPPORTED, w + ": fp32 or bf16 tensors");
    if (l.master(i) && l.types[i] != TSP_BF16) return fail(TSP_ERR_INVALID_ARG, w + ": a master beside an fp32 weight");
    if (!l.params[i] || !l.m[i] || !l.v[i] || (l.bits == 8 && (!l.ms[i] || !l.vs[i])))
      return fail(TSP_ERR_INVALID_ARG, w + ": null tensor");
    auto off = [](const void* p, unsigned a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
    const unsigned sa = l.bits == 32 ? 4u : 1u;
    if (off(l.params[i], l.types[i] == TSP_F32 ? 4u : 2u) || off(l.grads[i], l.grad_types[i] == TSP_F32 ? 4u : 2u) ||
        off(l.master(i), 4) || off(l.m[i], sa) || off(l.v[i], sa) || (l.bits == 8 && (off(l.ms[i], 4) || off(l.vs[i], 4))))
      return fail(TSP_ERR_INVALID_ARG, w + ": tensor not aligned to its element");
  }
  if (total >= (1ll << 31)) return fail(TSP_ERR_UNSUPPORTED, w + ": too many elements");
  return TSP_OK;
}

// What the step writes may not overlap anything else that it reads or writes.
tsp_status check_overlap(const char* what, const List& l) {
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  std::vector<Range> r;
  r.reserve(7 * (size_t)l.n);
  auto add = [&](const void* p, uint64_t bytes, bool out) {
    if (p) r.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, out});
  };
  for (int i = 0; i < l.n; ++i) {
    if (l.skipped(i)) continue;
    const uint64_t n = (uint64_t)l.sizes[i], state = l.bits == 32 ? 4 * n : n;
    add(l.params[i], n * (l.types[i] == TSP_F32 ? 4u : 2u), true);
    add(l.master(i), 4 * n, true);
    add(l.grads[i], n * (l.grad_types[i] == TSP_F32 ? 4u : 2u), false);
    add(l.m[i], state, true);
    add(l.v[i], state, true);
    if (l.bits == 8) {
      add(l.ms[i], 4 * ((n + 127) / 128), true);
      add(l.vs[i], 4 * ((n + 127) / 128), true);
    }
  }
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
  uintptr_t out_end = 0, any_end = 0;
  for (const Range& x : r) {
    if (x.lo < out_end || (x.out && x.lo < any_end))
      return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": a weight or state overlaps another tensor");
    if (x.out) out_end = std::max(out_end, x.hi);
    any_end = std::max(any_end, x.hi);
  }
  return TSP_OK;
}

template <int N, bool STATE8, bool FULL_RANGE>
tsp_status run(const List& l, const Step& a, cudaStream_t s) {
  static_assert(sizeof(Table<N>) + sizeof(Step) <= 32 * 1024 - 4, "kernel parameters");
  Table<N> t;
  t.count = 0;
  auto flush = [&](unsigned int chunks) -> tsp_status {
    if (t.count == 0) return TSP_OK;
    t.first[t.count] = chunks;
    adamw_kernel<N, STATE8, FULL_RANGE><<<chunks, kThreads, 0, s>>>(t, a);
    const cudaError_t e = cudaGetLastError();
    t.count = 0;
    return e == cudaSuccess ? TSP_OK : cuda_fail(e, "adamw: launch");
  };
  unsigned int chunk = 0;
  for (int i = 0; i < l.n; ++i) {
    // the random bits go by a tensor's place in the list, which is index0 + k: a launch ends where
    // a tensor without a gradient lies between two others
    if (t.count && (t.count == N || t.index0 + t.count != i)) TSP_TRY(flush(chunk));
    if (l.skipped(i)) continue;
    if (t.count == 0) {
      t.index0 = i;
      chunk = 0;
    }
    const int k = t.count++;
    const bool master = l.master(i) != nullptr;
    t.p[k] = master ? l.master(i) : l.params[i];
    t.p16[k] = master ? l.params[i] : nullptr;
    t.g[k] = l.grads[i];
    t.m[k] = l.m[i];
    t.v[k] = l.v[i];
    t.ms[k] = STATE8 ? l.ms[i] : nullptr;
    t.vs[k] = STATE8 ? l.vs[i] : nullptr;
    t.n[k] = (unsigned long long)l.sizes[i];
    t.first[k] = chunk;
    chunk += (unsigned int)((l.sizes[i] + kChunk - 1) / kChunk);
    uintptr_t low = reinterpret_cast<uintptr_t>(t.p16[k]) * 2;
    low |= l.types[i] == TSP_BF16 && !master ? reinterpret_cast<uintptr_t>(t.p[k]) * 2 : reinterpret_cast<uintptr_t>(t.p[k]);
    low |= reinterpret_cast<uintptr_t>(t.g[k]) * (l.grad_types[i] == TSP_BF16 ? 2 : 1);
    low |= (reinterpret_cast<uintptr_t>(t.m[k]) | reinterpret_cast<uintptr_t>(t.v[k])) * (STATE8 ? 4 : 1);
    t.kind[k] = (l.grad_types[i] == TSP_BF16 ? GRAD_BF16 : 0) | (l.types[i] == TSP_BF16 && !master ? PARAM_BF16 : 0) |
                (master ? MASTER : 0) | (low % 16 == 0 ? ALIGNED : 0);
  }
  return flush(chunk);
}

}  // namespace
}  // namespace tsp

using namespace tsp;

namespace tsp {
namespace {

tsp_status check_step(const char* what, const tsp_adamw* step, const List& l) {
  const std::string w(what);
  if (!step) return fail(TSP_ERR_INVALID_ARG, w + ": null step");
  const tsp_adamw& h = *step;
  if (!(h.beta1 >= 0. && h.beta1 < 1.) || !(h.beta2 >= 0. && h.beta2 < 1.))
    return fail(TSP_ERR_INVALID_ARG, w + ": betas in [0, 1)");
  // the approximate quotient takes no smaller divisor
  if (!((float)h.eps >= 1.17549435e-38f) || !std::isfinite(h.eps))
    return fail(TSP_ERR_INVALID_ARG, w + ": eps must be finite and at least 2^-126");
  if (!h.device_lr && !(h.lr >= 0. && std::isfinite(h.lr))) return fail(TSP_ERR_INVALID_ARG, w + ": lr must be finite, not negative");
  if (!(h.weight_decay >= 0.) || !std::isfinite(h.weight_decay))
    return fail(TSP_ERR_INVALID_ARG, w + ": weight_decay must be finite, not negative");
  if (!h.device_t && h.t < 1) return fail(TSP_ERR_INVALID_ARG, w + ": steps count from 1");
  if (h.norm && !(h.max_norm >= 0.)) return fail(TSP_ERR_INVALID_ARG, w + ": max_norm must not be negative");
  if (reinterpret_cast<uintptr_t>(h.norm) % 4 || reinterpret_cast<uintptr_t>(h.device_lr) % 4 ||
      reinterpret_cast<uintptr_t>(h.device_t) % 8)
    return fail(TSP_ERR_INVALID_ARG, w + ": norm, device_lr or device_t is misaligned");
  TSP_TRY(check_list(what, l));
  return check_overlap(what, l);
}

}  // namespace
}  // namespace tsp

extern "C" {

tsp_status tsp_adamw_check(int n, void* const* params, const int* types, void* const* masters,
                           const void* const* grads, const int* grad_types, void* const* m, void* const* v,
                           float* const* m_scales, float* const* v_scales, const int64_t* sizes, int state_bits,
                           const tsp_adamw* step) {
  TSP_GUARD_BEGIN
  return check_step("tsp_adamw_check", step,
                    {n, params, types, masters, grads, grad_types, m, v, m_scales, v_scales, sizes, state_bits});
  TSP_GUARD_END
}

tsp_status tsp_adamw_step(int n, void* const* params, const int* types, void* const* masters,
                          const void* const* grads, const int* grad_types, void* const* m, void* const* v,
                          float* const* m_scales, float* const* v_scales, const int64_t* sizes, int state_bits,
                          const tsp_adamw* step, void* stream) {
  TSP_GUARD_BEGIN
  const List l{n, params, types, masters, grads, grad_types, m, v, m_scales, v_scales, sizes, state_bits};
  TSP_TRY(check_step("tsp_adamw_step", step, l));
  const tsp_adamw& h = *step;
  const double log1 = std::log(h.beta1), log2 = std::log(h.beta2);
  const Step a{(float)h.beta1, (float)h.beta2, (float)(1. - h.beta1), (float)(1. - h.beta2), (float)h.eps,
               (float)(h.lr / -std::expm1((double)h.t * log1)), (float)(1. / std::sqrt(-std::expm1((double)h.t * log2))),
               (float)(h.lr * h.weight_decay), (float)h.max_norm, h.lr, h.weight_decay, log1, log2, (long long)h.t,
               h.seed, h.norm, h.device_lr, reinterpret_cast<const long long*>(h.device_t)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // With 8-bit states, whose kernel is bound by its instructions, numbers below 2^-126 count as 0 in root and quotient
  // where eps is so far above that it does not show: the root, at most 2^-63 / sqrt(1 - beta2^t), is below 2^-24 of eps,
  // and a step that is lost, below 2^-126 / eps, below 2^-87. 202M weights with masters 632 us, and 655 with a smaller
  // eps. With 32-bit states every number counts: 866 us either way.
  const bool full = !(h.eps >= std::ldexp(1. / std::sqrt(1. - h.beta2), -39));
  auto small = state_bits == 32 ? run<kSmall, false, true> : full ? run<kSmall, true, true> : run<kSmall, true, false>;
  auto large = state_bits == 32 ? run<kLarge, false, true> : full ? run<kLarge, true, true> : run<kLarge, true, false>;
  return (n <= kSmall ? small : large)(l, a, s);
  TSP_GUARD_END
}

}  // extern "C"
