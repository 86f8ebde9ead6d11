// Norm of many gradient tensors and clipping.
#include <cuda_fp16.h>

#include "../../include/mi_block.h"
#include "mi_internal.h"
#include "ptx.cuh"

namespace mi {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kItem = 2048;     // elements that a warp takes at a time
constexpr int kTable = 1000;    // tensors of one launch: their table is a kernel parameter (up to 32,764 bytes)

// A launch's tensors; tensor i has items [first[i], first[i + 1]).
struct Entry {
  const void* grad;
  void* out;
  long long count;
  uint32_t first;
  int dtype;
};
struct Table {
  int n;
  uint32_t items;
  Entry e[kTable];
};

// The tensor that item i belongs to.
__device__ __forceinline__ int tensor_of(const Table& t, uint32_t item) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= item) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float load(const void* p, int dtype, long long i) {
  if (dtype == MI_F32) return static_cast<const float*>(p)[i];
  if (dtype == MI_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void store(void* p, int dtype, long long i, float v) {
  if (dtype == MI_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == MI_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// partial[CTA] = the sum of the squares of the CTA's items, in 64 bits.  A lane squares and adds 64 elements in 32 bits; a
// sum that may have left that range is taken again with the elements scaled by a power of two.
__global__ void __launch_bounds__(kThreads) grad_square_kernel(const __grid_constant__ Table t, double* partial) {
  __shared__ double sums[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double acc = 0.0;
  for (uint32_t item = blockIdx.x * kWarps + warp; item < t.items; item += gridDim.x * kWarps) {
    const Entry& e = t.e[tensor_of(t, item)];
    const long long i0 = (long long)(item - e.first) * kItem;
    const long long i1 = i0 + kItem < e.count ? i0 + kItem : e.count;
    float s = 0.0f;
    for (long long i = i0 + lane; i < i1; i += 32) {
      const float v = load(e.grad, e.dtype, i);
      s = fmaf(v, v, s);
    }
    if (s > 0x1p-80f && s < 0x1p120f) {
      acc += (double)s;
    } else {
      const float up = s <= 0x1p-80f ? 0x1p100f : 0x1p-100f;
      float z = 0.0f;
      for (long long i = i0 + lane; i < i1; i += 32) {
        const float v = load(e.grad, e.dtype, i) * up;
        z = fmaf(v, v, z);
      }
      acc += (double)z * (s <= 0x1p-80f ? 0x1p-200 : 0x1p200);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    partial[blockIdx.x] = total;
  }
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const double* partial, int n, float* norm) {
  grid_dep_wait();
  grid_dep_launch();
  double t = 0.0;
  for (int i = threadIdx.x; i < n; i += 32) t += partial[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(t);
}

// min(1, max_norm / (norm + 1e-6)); a NaN stays one.
__device__ __forceinline__ float clip_factor(float max_norm, float norm) {
  const float q = max_norm / (norm + 1e-6f);
  return q >= 1.0f ? 1.0f : q;
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Table t, const float* norm,
                                                              float max_norm) {
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float c = clip_factor(max_norm, norm[0]);
  for (uint32_t item = blockIdx.x * kWarps + warp; item < t.items; item += gridDim.x * kWarps) {
    const Entry& e = t.e[tensor_of(t, item)];
    if (c == 1.0f && e.grad == e.out) continue;
    const long long i0 = (long long)(item - e.first) * kItem;
    const long long i1 = i0 + kItem < e.count ? i0 + kItem : e.count;
    for (long long i = i0 + lane; i < i1; i += 32) store(e.out, e.dtype, i, load(e.grad, e.dtype, i) * c);
  }
}

// Takes tensors from `at` on into a table, as many as one launch holds; returns the next.
int fill(const GradTensor* g, int n, int at, Table* t) {
  t->n = 0;
  uint64_t items = 0;
  for (; at < n && t->n < kTable; ++at) {
    if (g[at].count == 0) continue;
    const uint64_t mine = (uint64_t)(g[at].count + kItem - 1) / kItem;
    if (t->n > 0 && items + mine > 0x40000000u) break;
    t->e[t->n++] = Entry{g[at].grad, g[at].out, g[at].count, (uint32_t)items, g[at].dtype};
    items += mine;
  }
  t->items = (uint32_t)items;
  return at;
}

int grid_of(uint32_t items, int num_sms) {
  const uint32_t need = (items + kWarps - 1) / kWarps, cap = 2 * (uint32_t)num_sms;
  return (int)(need < cap ? need : cap);
}

}  // namespace

size_t grads_workspace(const GradTensor* g, int n, int num_sms) {
  size_t ctas = 0;
  Table t;
  for (int at = 0; at < n;) {
    at = fill(g, n, at, &t);
    ctas += grid_of(t.items, num_sms);
  }
  return ctas * sizeof(double);
}

cudaError_t grads_launch(const GradTensor* g, int n, bool compute, bool clip, float max_norm, float* norm, void* ws,
                         int num_sms, cudaStream_t s) {
  double* partial = static_cast<double*>(ws);
  Table t;
  cudaError_t e;
  if (compute) {
    int ctas = 0;
    for (int at = 0; at < n;) {
      at = fill(g, n, at, &t);
      const int grid = grid_of(t.items, num_sms);
      if (grid == 0) continue;
      e = launch_kernel(grad_square_kernel, dim3(grid), dim3(kThreads), 0, s, true, t, partial + ctas);
      if (e != cudaSuccess) return e;
      ctas += grid;
    }
    e = launch_kernel(grad_norm_kernel, dim3(1), dim3(32), 0, s, true, (const double*)partial, ctas, norm);
    if (e != cudaSuccess) return e;
  }
  if (!clip) return cudaSuccess;
  for (int at = 0; at < n;) {
    at = fill(g, n, at, &t);
    const int grid = grid_of(t.items, num_sms);
    if (grid == 0) continue;
    e = launch_kernel(grad_scale_kernel, dim3(grid), dim3(kThreads), 0, s, true, t, (const float*)norm, max_norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mi
