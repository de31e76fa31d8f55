// grad_clip.cu - the global 2-norm of a list of gradient tensors, and their scaling to a
// largest norm:
//     norm = sqrt(sum over all tensors and elements of g^2)
//     out  = g * min(1, max_norm / (norm + 1e-6))
//
// Bound: HBM. The norm reads every gradient once; the scaling reads it again and writes
// it. The list travels in the kernels' parameters (no copy to the device, so the calls
// can be captured), 64 or 1024 tensors per launch, cut into chunks of 16384 elements
// that persistent CTAs take in turn; a chunk's tensor is found by a binary search over
// the first chunk of each tensor. The scaling walks the chunks backwards, because the
// end of the list is what the norm has left in L2.
//
// Sums: 64 squares per thread and chunk in fp32, in four chains of at most 17, then fp64 over
// chunks, threads, CTAs and launches, each in a fixed order, so a result does not change from run
// to run. Tensors that do not start on 16 bytes take single elements up to the boundary and 16
// bytes at a time from there (norm of 100M elements, aligned and one element off: fp32 66 and 71
// us, bf16 38 and 43). A thread whose fp32 sum overflowed, or is so small that squares may have
// vanished, takes its elements again in fp64: the norm holds over the whole range of
// fp32 gradients.
#include <algorithm>
#include <cmath>
#include <vector>

#include "tsp_device.cuh"
#include "tsp_internal.h"

namespace tsp {
namespace {

constexpr int kChunk = 16384;
constexpr int kThreads = 256;
constexpr int kCtas = 608;   // partial sums per launch: a constant, so that their order is
constexpr int kSmall = 64;   // tensors per launch in the small table (1.9 KB of parameters)
constexpr int kLarge = 1024; // and in the large one

template <int N>
struct Table {
  const void* in[N];
  void* out[N];
  unsigned long long n[N];     // elements
  unsigned int first[N + 1];   // first chunk
  unsigned char bf16[N];
  int count;
};

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, unsigned int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {  // the last tensor whose first chunk is not behind `chunk`
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool vec_ok(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Elements of the n at p before the first 16-byte boundary.
template <class E>
__device__ __forceinline__ int elements_ahead(const E* p, int n) {
  return min(n, (int)((0u - (unsigned)reinterpret_cast<uintptr_t>(p)) & 15u) / (int)sizeof(E));
}

// f(v, chain) for each of this thread's elements of the chunk [p, p + n): 16 bytes at a time
// between the boundaries, single elements at the two ends, those in chains of their own.
template <class F>
__device__ __forceinline__ void each_f32(const float* p, int n, F f) {
  const int ahead = elements_ahead(p, n);
  if (threadIdx.x < ahead) f(p[threadIdx.x], 1);
  p += ahead;
  n -= ahead;
  const float4* q = reinterpret_cast<const float4*>(p);
  const int nv = n >> 2;
  int i = threadIdx.x;
  for (; i + 3 * kThreads < nv; i += 4 * kThreads) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = q[i + k * kThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k) f(v[k].x, 0), f(v[k].y, 1), f(v[k].z, 2), f(v[k].w, 3);
  }
  for (; i < nv; i += kThreads) {
    const float4 v = q[i];
    f(v.x, 0), f(v.y, 1), f(v.z, 2), f(v.w, 3);
  }
  for (int j = (nv << 2) + threadIdx.x; j < n; j += kThreads) f(p[j], 0);
}

template <class F>
__device__ __forceinline__ void each_bf16(const __nv_bfloat16* p, int n, F f) {
  const int ahead = elements_ahead(p, n);
  if (threadIdx.x < ahead) f(__bfloat162float(p[threadIdx.x]), 1);
  p += ahead;
  n -= ahead;
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const int nv = n >> 3;
  int i = threadIdx.x;
  for (; i + 3 * kThreads < nv; i += 4 * kThreads) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = q[i + k * kThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f(bf16_lo(v[k].x), 0), f(bf16_hi(v[k].x), 1), f(bf16_lo(v[k].y), 2), f(bf16_hi(v[k].y), 3);
      f(bf16_lo(v[k].z), 0), f(bf16_hi(v[k].z), 1), f(bf16_lo(v[k].w), 2), f(bf16_hi(v[k].w), 3);
    }
  }
  for (; i < nv; i += kThreads) {
    const uint4 v = q[i];
    f(bf16_lo(v.x), 0), f(bf16_hi(v.x), 1), f(bf16_lo(v.y), 2), f(bf16_hi(v.y), 3);
    f(bf16_lo(v.z), 0), f(bf16_hi(v.z), 1), f(bf16_lo(v.w), 2), f(bf16_hi(v.w), 3);
  }
  for (int j = (nv << 3) + threadIdx.x; j < n; j += kThreads) f(__bfloat162float(p[j]), 0);
}

template <class F>
__device__ __forceinline__ void each(const void* p, bool bf16, unsigned long long at, int n, F f) {
  if (bf16) each_bf16(static_cast<const __nv_bfloat16*>(p) + at, n, f);
  else each_f32(static_cast<const float*>(p) + at, n, f);
}

// Sum over the block in a fixed order; valid in every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) s += part[k];
  return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4)
    grad_norm_kernel(const __grid_constant__ Table<N> t, double* partial) {
  double sum = 0.;
  dependents_may_start();
  const unsigned int chunks = t.first[t.count];
  for (unsigned int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const unsigned long long at = (unsigned long long)(c - t.first[i]) * kChunk;
    const int n = (int)min((unsigned long long)kChunk, t.n[i] - at);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t bits = 0;
    each(t.in[i], t.bf16[i], at, n, [&](float g, int k) {
      acc[k] = fmaf(g, g, acc[k]);
      bits |= __float_as_uint(g);
    });
    const float s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    double d = (double)s;
    // above 2^-60 the squares that vanished (below 2^-149 each) are under 2^-80 of the sum
    if (!(s < 3.0e38f) || (s < 8.7e-19f && (bits & 0x7fffffffu) != 0u)) {
      d = 0.;
      each(t.in[i], t.bf16[i], at, n, [&](float g, int) { d += (double)g * (double)g; });
    }
    sum += d;
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the partial sums, the same bits in every block.
__device__ __forceinline__ double norm_of(const double* partial, int n) {
  double s = 0.;
  prior_kernel_done();
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  return sqrt(block_sum(s));
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(const double* partial, int n,
                                                                  float* norm) {
  const double v = norm_of(partial, n);
  if (threadIdx.x == 0) *norm = (float)v;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4)
    grad_scale_kernel(const __grid_constant__ Table<N> t, const double* partial, int n_partial,
                      float max_norm, float* norm) {
  const double v = norm_of(partial, n_partial);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  // an infinite max_norm clips nothing, not even an infinite norm; a NaN norm stays one
  const double want = isinf(max_norm) && !isnan(v) ? 1. : (double)max_norm / (v + 1e-6);
  // a NaN norm gives a NaN factor; one below 2^-100, which fp32 would round to few bits,
  // is applied as factor * 2^64 and then 2^-64, which is exact
  const bool tiny = want < 7.9e-31;
  const float factor = want >= 1. ? 1.f : (float)(tiny ? want * 18446744073709551616. : want);
  const float rest = tiny ? 5.4210108624275222e-20f : 1.f;
  const unsigned int chunks = t.first[t.count];
  for (unsigned int k = blockIdx.x; k < chunks; k += gridDim.x) {
    const unsigned int c = chunks - 1 - k;
    const int i = tensor_of(t, c);
    if (factor == 1.f && t.in[i] == t.out[i]) continue;
    const unsigned long long at = (unsigned long long)(c - t.first[i]) * kChunk;
    const int n = (int)min((unsigned long long)kChunk, t.n[i] - at);
    if (t.bf16[i]) {
      const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(t.in[i]) + at;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(t.out[i]) + at;
      int j = threadIdx.x;
      if (vec_ok(in) && vec_ok(out)) {
        const uint4* q = reinterpret_cast<const uint4*>(in);
        uint4* o = reinterpret_cast<uint4*>(out);
        auto scaled = [&](uint32_t u) { return pack_bf16x2(bf16_lo(u) * factor * rest, bf16_hi(u) * factor * rest); };
        for (; j < (n >> 3); j += kThreads) {
          const uint4 u = q[j];
          o[j] = make_uint4(scaled(u.x), scaled(u.y), scaled(u.z), scaled(u.w));
        }
        j = (n >> 3 << 3) + threadIdx.x;
      }
      for (; j < n; j += kThreads) out[j] = __float2bfloat16_rn(__bfloat162float(in[j]) * factor * rest);
    } else {
      const float* in = static_cast<const float*>(t.in[i]) + at;
      float* out = static_cast<float*>(t.out[i]) + at;
      int j = threadIdx.x;
      if (vec_ok(in) && vec_ok(out)) {
        const float4* q = reinterpret_cast<const float4*>(in);
        float4* o = reinterpret_cast<float4*>(out);
        const int nv = n >> 2;
        for (; j + 3 * kThreads < nv; j += 4 * kThreads) {
          float4 u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = q[j + e * kThreads];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[j + e * kThreads] = make_float4(u[e].x * factor * rest, u[e].y * factor * rest,
                                            u[e].z * factor * rest, u[e].w * factor * rest);
        }
        for (; j < nv; j += kThreads) {
          const float4 u = q[j];
          o[j] = make_float4(u.x * factor * rest, u.y * factor * rest, u.z * factor * rest,
                             u.w * factor * rest);
        }
        j = (nv << 2) + threadIdx.x;
      }
      for (; j < n; j += kThreads) out[j] = in[j] * factor * rest;
    }
  }
}

struct List {
  int n;
  const void* const* in;
  void* const* out;
  const int64_t* sizes;
  const int* types;
};

// Tensors [i0, i0 + count) of the list as a kernel parameter.
template <int N>
void fill(Table<N>& t, const List& l, int i0, int count) {
  unsigned int chunk = 0;
  t.count = count;
  for (int k = 0; k < count; ++k) {
    t.in[k] = l.in[i0 + k];
    t.out[k] = l.out ? l.out[i0 + k] : nullptr;
    t.n[k] = (unsigned long long)l.sizes[i0 + k];
    t.bf16[k] = l.types[i0 + k] == TSP_BF16;
    t.first[k] = chunk;
    chunk += (unsigned int)((l.sizes[i0 + k] + kChunk - 1) / kChunk);
  }
  t.first[count] = chunk;
}

int launches_of(int n) { return n <= kSmall ? 1 : (n + kLarge - 1) / kLarge; }

template <int N>
tsp_status run(const List& l, double* partial, float max_norm, float* norm, cudaStream_t s) {
  const int launches = launches_of(l.n);
  const int n_partial = launches * kCtas;
  static_assert(sizeof(Table<N>) <= 32 * 1024, "kernel parameters");
  Table<N> t;
  for (int k = 0; k < launches; ++k) {
    fill(t, l, k * N, std::min(N, l.n - k * N));
    grad_norm_kernel<N><<<kCtas, kThreads, 0, s>>>(t, partial + (size_t)k * kCtas);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "gradient clip: launch");
  if (!l.out) {
    e = launch_early(grad_norm_join_kernel, 1, kThreads, 0, s, partial, n_partial, norm);
    return e == cudaSuccess ? TSP_OK : cuda_fail(e, "gradient norm: launch");
  }
  for (int k = launches - 1; k >= 0; --k) {
    if (launches > 1) fill(t, l, k * N, std::min(N, l.n - k * N));
    const unsigned int ctas = std::max(1u, std::min((unsigned)kCtas, t.first[t.count]));
    if (k == launches - 1) {
      e = launch_early(grad_scale_kernel<N>, ctas, kThreads, 0, s, t, partial, n_partial, max_norm, norm);
    } else {
      grad_scale_kernel<N><<<ctas, kThreads, 0, s>>>(t, partial, n_partial, max_norm, norm);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return cuda_fail(e, "gradient clip: launch");
  }
  return TSP_OK;
}

tsp_status check_list(const char* what, const List& l, const float* norm, void* ws) {
  const std::string w(what);
  if (l.n < 0 || l.n > TSP_GRAD_MAX_TENSORS)
    return fail(TSP_ERR_UNSUPPORTED, w + ": 0 to 65536 tensors");
  if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u))
    return fail(TSP_ERR_INVALID_ARG, w + ": norm is null or misaligned");
  TSP_TRY(check_ws(ws, what));
  if (l.n && (!l.in || !l.sizes || !l.types)) return fail(TSP_ERR_INVALID_ARG, w + ": null list");
  for (int i = 0; i < l.n; ++i) {
    if (l.types[i] != TSP_F32 && l.types[i] != TSP_BF16)
      return fail(TSP_ERR_UNSUPPORTED, w + ": fp32 or bf16 tensors");
    const unsigned a = l.types[i] == TSP_F32 ? 4u : 2u;
    if (l.sizes[i] < 0 || l.sizes[i] > (1ll << 40))
      return fail(TSP_ERR_INVALID_ARG, w + ": tensor size out of range");
    if (l.sizes[i] == 0) continue;
    if (!l.in[i] || (l.out && !l.out[i])) return fail(TSP_ERR_INVALID_ARG, w + ": null tensor");
    if (reinterpret_cast<uintptr_t>(l.in[i]) % a || (l.out && reinterpret_cast<uintptr_t>(l.out[i]) % a))
      return fail(TSP_ERR_INVALID_ARG, w + ": tensor not aligned to its element");
  }
  // at most 2^31 chunks (2^45 elements) over the list, so that a launch's chunk numbers and its
  // stride of CTAs fit 32 bits
  int64_t total = 0;
  for (int i = 0; i < l.n; ++i) total += (l.sizes[i] + kChunk - 1) / kChunk;
  if (total > (1ll << 31)) return fail(TSP_ERR_UNSUPPORTED, w + ": too many elements");
  return TSP_OK;
}

// No output may overlap another output or another tensor's input: the scaling would read
// or write it twice. An output may be its own input.
tsp_status check_overlap(const char* what, const List& l) {
  struct Range {
    uintptr_t lo, hi;
    int i;
    bool out;
  };
  std::vector<Range> r;
  r.reserve(2 * (size_t)l.n);
  for (int i = 0; i < l.n; ++i) {
    const uintptr_t bytes = (uintptr_t)l.sizes[i] * (l.types[i] == TSP_F32 ? 4u : 2u);
    if (!bytes) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(l.in[i]), b = reinterpret_cast<uintptr_t>(l.out[i]);
    r.push_back({b, b + bytes, i, true});
    if (a != b) r.push_back({a, a + bytes, i, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
  // the furthest end so far of an output and of any range: a range that starts before the
  // former overlaps an output, an output that starts before the latter overlaps something
  uintptr_t out_end = 0, any_end = 0;
  for (const Range& x : r) {
    if (x.lo < out_end || (x.out && x.lo < any_end))
      return fail(TSP_ERR_INVALID_ARG, std::string(what) + ": an output overlaps another tensor");
    if (x.out) out_end = std::max(out_end, x.hi);
    any_end = std::max(any_end, x.hi);
  }
  return TSP_OK;
}

tsp_status norm_and_scale(const List& l, float max_norm, float* norm, void* ws, cudaStream_t s) {
  double* partial = static_cast<double*>(ws);
  if (l.n <= kSmall) return run<kSmall>(l, partial, max_norm, norm, s);
  return run<kLarge>(l, partial, max_norm, norm, s);
}

}  // namespace
}  // namespace tsp

using namespace tsp;

extern "C" {

size_t tsp_grad_workspace_bytes(int n) {
  if (n < 0 || n > TSP_GRAD_MAX_TENSORS) return 0;
  return align256((size_t)(n ? launches_of(n) : 1) * kCtas * sizeof(double));
}

tsp_status tsp_grad_norm(int n, const void* const* grads, const int64_t* sizes, const int* types,
                         float* norm, void* ws, void* stream) {
  TSP_GUARD_BEGIN
  const List l{n, grads, nullptr, sizes, types};
  TSP_TRY(check_list("tsp_grad_norm", l, norm, ws));
  return norm_and_scale(l, 0.f, norm, ws, static_cast<cudaStream_t>(stream));
  TSP_GUARD_END
}

tsp_status tsp_grad_clip(int n, const void* const* grads, void* const* outs, const int64_t* sizes,
                         const int* types, float max_norm, float* norm, void* ws, void* stream) {
  TSP_GUARD_BEGIN
  if (n > 0 && !outs) return fail(TSP_ERR_INVALID_ARG, "tsp_grad_clip: null list");
  if (!(max_norm >= 0.f)) return fail(TSP_ERR_INVALID_ARG, "tsp_grad_clip: max_norm must not be negative");
  const void* none = nullptr;
  void* none_out = nullptr;
  const List l{n, n > 0 ? grads : &none, n > 0 ? outs : &none_out, sizes, types};
  TSP_TRY(check_list("tsp_grad_clip", l, norm, ws));
  TSP_TRY(check_overlap("tsp_grad_clip", l));
  return norm_and_scale(l, max_norm, norm, ws, static_cast<cudaStream_t>(stream));
  TSP_GUARD_END
}

}  // extern "C"
