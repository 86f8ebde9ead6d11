// Norm of many gradient tensors and clipping.
//
// Both are bound by HBM: the norm reads every gradient once; clipping needs the norm of all of them first, so it reads
// them again, and writes them.  A set's tensors are cut into items of 256 vectors of 16 bytes (4 KB: 8 loads in flight a
// lane, which with 32 warps per SM is 128 KB on the way), a CTA takes a contiguous range of items and its warps every 8th of
// it.  The norm walks the ranges upwards and the clipping downwards: what the norm has read last is still in the L2 cache, all
// of a set that fits it.  Which tensor an item belongs to comes from a table that is a kernel parameter: there is no
// device memory to keep or to fill, and a captured graph holds its own copy.
//
// A tensor may begin anywhere: the elements in front of its first and behind its last 16-byte boundary go with its first and
// last item, one by one.  Where a gradient and the tensor that takes it clipped lie differently to those boundaries, the
// clipping goes element by element.
#include <algorithm>

#include "../../include/mi_block.h"
#include "mi_internal.h"
#include "ptx.cuh"
#include "values.cuh"

namespace mi {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 4;     // per SM
constexpr int kVectors = 8;  // a lane's of an item
constexpr float kSmallest = 0x1p-80f, kLargest = 0x1p120f;

// The tensor that `item` belongs to.
__device__ __forceinline__ int tensor_of(const GradEntry* e, int n, uint32_t item) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid].first <= item) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One item of a tensor: `vectors` of 16 bytes from the element `at` on, and `head` elements in front of the tensor's first
// one and `tail` behind its last.
struct Item {
  int vectors, head, tail;
  long long at, tail_at;
  __device__ __forceinline__ Item(const GradEntry& e, uint32_t item, int size) {
    const int per = 16 / size;
    const long long lead = min((long long)((0u - (uint32_t)reinterpret_cast<uintptr_t>(e.grad)) & 15u) / size, e.count);
    const long long all = (e.count - lead) / per, v0 = (long long)(item - e.first) * (32 * kVectors);
    vectors = (int)min(all - v0, 32LL * kVectors);
    at = lead + v0 * per;
    head = item == e.first ? (int)lead : 0;
    tail_at = lead + all * per;
    tail = v0 + 32 * kVectors >= all ? (int)(e.count - tail_at) : 0;
  }
};

__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// A vector as pairs in fp32, and back (rounded once).
template <typename T> struct Vec {
  static constexpr int N = 4;
  __device__ __forceinline__ static void unpack(const uint4& v, f32x2_t (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = unpack2<T>(w[i]);
  }
  __device__ __forceinline__ static uint4 pack(const f32x2_t (&f)[4]) {
    return make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
  }
};
template <> struct Vec<float> {
  static constexpr int N = 2;
  __device__ __forceinline__ static void unpack(const uint4& v, f32x2_t (&f)[2]) {
    f[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ static uint4 pack(const f32x2_t (&f)[2]) {
    float a, b, c, d;
    f2_unpack(f[0], a, b);
    f2_unpack(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
};

// An item whose squares may leave fp32's range, again: a lane's elements times a power of two, whose square the sum is
// divided by.  top: the warp's largest sum as it was (infinity for NaN; 0 where all were too small).
__device__ __noinline__ double item_squares_scaled(const void* grad, int dtype, long long i0, long long i1, float top) {
  const float up = top <= kSmallest ? 0x1p100f : 0x1p-100f;
  float z = 0.0f;
  for (long long i = i0 + (threadIdx.x & 31); i < i1; i += 32) {
    const float v = value_at(grad, dtype, i, 0.0f) * up;
    z = fmaf(v, v, z);
  }
  return (double)z * (top <= kSmallest ? 0x1p-200 : 0x1p200);  // (NaN stays)
}

// A lane's part of an item's sum of squares, in 64 bits.  Up to 65 squares are added in 32 bits; where a lane's sum may have
// left that range (a square overflows from 2^64 on and loses bits below 2^-63) the warp takes the item again, scaled.
template <typename T>
__device__ __forceinline__ double item_squares(const GradEntry& e, uint32_t item) {
  const int lane = threadIdx.x & 31;
  const Item t(e, item, sizeof(T));
  const T* g = static_cast<const T*>(e.grad);
  const uint4* from = reinterpret_cast<const uint4*>(g + t.at) + lane;
  uint4 v[kVectors];
#pragma unroll
  for (int k = 0; k < kVectors; ++k) v[k] = k * 32 + lane < t.vectors ? __ldcg(from + k * 32) : make_uint4(0, 0, 0, 0);
  float edge = 0.0f;  // an element outside of the vectors
  if (lane < t.head) edge = to_f32(g[lane]);
  else if (lane >= 16 && lane - 16 < t.tail) edge = to_f32(g[t.tail_at + lane - 16]);
  f32x2_t s2[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < kVectors; ++k) {
    f32x2_t f[Vec<T>::N];
    Vec<T>::unpack(v[k], f);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) s2[i & 1] = f2_fma(f[i], f[i], s2[i & 1]);
  }
  float lo, hi;
  f2_unpack(f2_add(s2[0], s2[1]), lo, hi);
  const float s = fmaf(edge, edge, lo + hi);
  if (__all_sync(0xffffffffu, s > kSmallest && s < kLargest)) return (double)s;
  const float low = s <= kSmallest ? 0.0f : s;  // the whole warp by its largest sum: small ones next to it do not count
  float top = low == low ? low : __int_as_float(0x7f800000);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top > 0.0f && top < kLargest) return (double)s;
  uint32_t bits = edge != 0.0f;
#pragma unroll
  for (int k = 0; k < kVectors; ++k) bits |= v[k].x | v[k].y | v[k].z | v[k].w;
  if (!__any_sync(0xffffffffu, bits != 0)) return 0.0;
  const long long i0 = t.head > 0 ? 0 : t.at, i1 = t.tail > 0 ? e.count : t.at + (long long)max(t.vectors, 0) * (16 / (int)sizeof(T));
  return item_squares_scaled(e.grad, e.dtype, i0, i1, top);
}

// Sum over the CTA in a fixed order, for thread 0.
__device__ __forceinline__ double cta_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += shared[w];
  return t;
}

// partial[CTA] = the sum of the squares of the CTA's items.
template <int kEntries>
__global__ void __launch_bounds__(kThreads, kCtas) grad_square_kernel(const __grid_constant__ GradTable<kEntries> t, double* partial) {
  __shared__ double sums[kWarps];
  const uint32_t i0 = (uint32_t)((uint64_t)t.items * blockIdx.x / gridDim.x), i1 = (uint32_t)((uint64_t)t.items * (blockIdx.x + 1) / gridDim.x);
  uint32_t item = i0 + (threadIdx.x >> 5);
  int at = item < i1 ? tensor_of(t.e, t.n, item) : 0;
  grid_dep_wait();
  grid_dep_launch();
  double acc = 0.0;
  for (; item < i1; item += kWarps) {
    while (at + 1 < t.n && t.e[at + 1].first <= item) ++at;
    const GradEntry& e = t.e[at];
    acc += e.dtype == MI_BF16 ? item_squares<__nv_bfloat16>(e, item)
           : e.dtype == MI_F32 ? item_squares<float>(e, item) : item_squares<__half>(e, item);
  }
  const double sum = cta_sum(acc, sums);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from n partial sums, the same in every CTA that asks.
__device__ __forceinline__ float norm_of(const double* partial, int n, double* shared) {
  double t = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) t += __ldcg(partial + i);
  return (float)sqrt(cta_sum(t, shared));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* partial, int n, float* norm) {
  __shared__ double sums[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const float v = norm_of(partial, n, sums);
  if (threadIdx.x == 0) norm[0] = v;
}

// min(1, max_norm / (norm + 1e-6)); a NaN stays one.
__device__ __forceinline__ float clip_factor(float max_norm, float norm) {
  const float q = max_norm / (norm + 1e-6f);
  return q >= 1.0f ? 1.0f : q;
}

__device__ __noinline__ void scale_elements(const GradEntry& e, long long i0, long long i1, float c) {
  for (long long i = i0 + (threadIdx.x & 31); i < i1; i += 32) {
    const float v = value_at(e.grad, e.dtype, i, 0.0f) * c;
    if (e.dtype == MI_F32) static_cast<float*>(e.out)[i] = v;
    else if (e.dtype == MI_F16) static_cast<__half*>(e.out)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(e.out)[i] = __float2bfloat16_rn(v);
  }
}

template <typename T>
__device__ __forceinline__ void scale_item(const GradEntry& e, uint32_t item, float c) {
  const int lane = threadIdx.x & 31;
  const Item t(e, item, sizeof(T));
  const T* g = static_cast<const T*>(e.grad);
  T* o = static_cast<T*>(e.out);
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15u) != 0) {
    scale_elements(e, t.head > 0 ? 0 : t.at, t.tail > 0 ? e.count : t.at + (long long)max(t.vectors, 0) * (16 / (int)sizeof(T)), c);
    return;
  }
  const uint4* from = reinterpret_cast<const uint4*>(g + t.at) + lane;
  uint4* to = reinterpret_cast<uint4*>(o + t.at) + lane;
  uint4 v[kVectors];
#pragma unroll
  for (int k = 0; k < kVectors; ++k)
    v[k] = k * 32 + lane < t.vectors ? from[k * 32] : make_uint4(0, 0, 0, 0);
  const f32x2_t cc = f2_of(c);
#pragma unroll
  for (int k = 0; k < kVectors; ++k) {
    f32x2_t f[Vec<T>::N];
    Vec<T>::unpack(v[k], f);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) f[i] = f2_mul(f[i], cc);
    // (evict-first: what is still to be read stays in the L2 cache)
    if (k * 32 + lane < t.vectors) __stcs(to + k * 32, Vec<T>::pack(f));
  }
  if (lane < t.head) from_f32(to_f32(g[lane]) * c, o[lane]);
  else if (lane >= 16 && lane - 16 < t.tail) from_f32(to_f32(g[t.tail_at + lane - 16]) * c, o[t.tail_at + lane - 16]);
}

// out = grad * factor.  parts > 0: the norm comes from that many partial sums, and CTA 0 of the first launch stores it.
template <int kEntries>
__global__ void __launch_bounds__(kThreads, kCtas) grad_scale_kernel(const __grid_constant__ GradTable<kEntries> t, const double* partial,
                                                                     int parts, float* norm, bool store, float max_norm) {
  __shared__ double sums[kWarps];
  const uint32_t i0 = (uint32_t)((uint64_t)t.items * blockIdx.x / gridDim.x), i1 = (uint32_t)((uint64_t)t.items * (blockIdx.x + 1) / gridDim.x);
  long long item = (long long)i1 - 1 - (threadIdx.x >> 5);
  int at = item >= (long long)i0 ? tensor_of(t.e, t.n, (uint32_t)item) : 0;
  grid_dep_wait();
  grid_dep_launch();
  float v;
  if (parts > 0) {
    v = norm_of(partial, parts, sums);
    if (store && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = v;
  } else {
    v = norm[0];
  }
  const float c = clip_factor(max_norm, v);
  for (; item >= (long long)i0; item -= kWarps) {
    while (t.e[at].first > (uint32_t)item) --at;
    const GradEntry& e = t.e[at];
    if (c == 1.0f && e.grad == e.out) continue;
    if (e.dtype == MI_BF16) scale_item<__nv_bfloat16>(e, (uint32_t)item, c);
    else if (e.dtype == MI_F32) scale_item<float>(e, (uint32_t)item, c);
    else scale_item<__half>(e, (uint32_t)item, c);
  }
}

int grid_of(uint32_t items, int num_sms) {
  const uint32_t need = (items + kWarps - 1) / kWarps, cap = (uint32_t)(kCtas * num_sms);
  return (int)(need < cap ? need : cap);
}

int grid_of(const GradPlan& p, size_t i, int num_sms) { return grid_of(p.small ? p.one.items : p.many[i].items, num_sms); }

}  // namespace

uint32_t grad_items(const GradEntry& e) {
  const long long size = e.dtype == MI_F32 ? 4 : 2;
  const long long lead = std::min((long long)((0u - (uint32_t)reinterpret_cast<uintptr_t>(e.grad)) & 15u) / size, e.count);
  const long long vectors = (e.count - lead) / (16 / size);
  return (uint32_t)std::max(1LL, (vectors + 32 * kVectors - 1) / (32 * kVectors));
}

size_t grads_workspace(const GradPlan& p, int num_sms) {
  size_t ctas = 0;
  for (size_t i = 0; i < p.launches(); ++i) ctas += grid_of(p, i, num_sms);
  return ctas * sizeof(double);
}

cudaError_t grads_launch(const GradPlan& p, bool compute, bool clip, float max_norm, float* norm, void* ws, int num_sms,
                         cudaStream_t s) {
  double* partial = static_cast<double*>(ws);
  int parts = 0;
  if (compute) {
    for (size_t i = 0; i < p.launches(); ++i) {
      const dim3 grid(grid_of(p, i, num_sms));
      const cudaError_t e =
          p.small ? launch_kernel(grad_square_kernel<kGradSmall>, grid, dim3(kThreads), 0, s, true, p.one, partial + parts)
                  : launch_kernel(grad_square_kernel<kGradLarge>, grid, dim3(kThreads), 0, s, true, p.many[i], partial + parts);
      if (e != cudaSuccess) return e;
      parts += (int)grid.x;
    }
    if (!clip || parts == 0) {
      const cudaError_t e = launch_kernel(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, true, (const double*)partial, parts, norm);
      if (e != cudaSuccess) return e;
    }
  }
  if (!clip) return cudaSuccess;
  for (size_t k = p.launches(); k > 0; --k) {  // (from the last one on: it was read last)
    const size_t i = k - 1;
    const dim3 grid(grid_of(p, i, num_sms));
    const cudaError_t e = p.small ? launch_kernel(grad_scale_kernel<kGradSmall>, grid, dim3(kThreads), 0, s, true, p.one,
                                                  (const double*)partial, parts, norm, true, max_norm)
                                  : launch_kernel(grad_scale_kernel<kGradLarge>, grid, dim3(kThreads), 0, s, true, p.many[i],
                                                  (const double*)partial, parts, norm, i == 0, max_norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mi
