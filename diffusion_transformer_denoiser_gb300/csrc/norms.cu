// Layer norm, its gradient, and the gradient of the modulated RMSNorm.
#include <cuda_fp16.h>

#include "../../include/mi_block.h"
#include "mi_internal.h"
#include "ptx.cuh"

namespace mi {

namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// Entry i of a parameter of the given type; p null: `none`.
__device__ __forceinline__ float param_at(const void* p, int dtype, long long i, float none) {
  if (p == nullptr) return none;
  if (dtype == MI_F32) return static_cast<const float*>(p)[i];
  if (dtype == MI_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sums over the CTA of two values, the same in every thread; s: 2 * kWarps floats of shared memory.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float2* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    t.x += s[w].x;
    t.y += s[w].y;
  }
  return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) layer_norm_kernel(LayerNormArgs a) {
  __shared__ float2 sums[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const float inv = 1.0f / (float)a.width;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (long long)row * a.x_stride;
    T* out = static_cast<T*>(a.out) + (long long)row * a.out_stride;
    float s = 0.0f, q = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) s += to_f32(x[c]);
    const float mean = cta_sum2(s, 0.0f, sums).x * inv;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      const float d = to_f32(x[c]) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = rsqrtf(cta_sum2(q, 0.0f, sums).x * inv + a.eps);
    for (int c = threadIdx.x; c < a.width; c += kThreads)
      from_f32(fmaf((to_f32(x[c]) - mean) * rstd, param_at(a.weight, a.param_dtype, c, 1.0f),
                    param_at(a.bias, a.param_dtype, c, 0.0f)), out[c]);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
  }
}

// A CTA takes a contiguous part of a group's rows and adds its columns' sums up in shared memory (a column belongs to one
// thread), then writes them to partial [group][part][2][width].
template <typename T, bool kRms>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(NormBwdArgs a, int parts) {
  extern __shared__ float acc[];  // [2][width]: sums of dy n and of dy
  __shared__ float2 sums[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const float inv = 1.0f / (float)a.width;
  const int group = blockIdx.x / parts, part = blockIdx.x % parts;
  const int r0 = (int)((long long)a.seq * part / parts), r1 = (int)((long long)a.seq * (part + 1) / parts);
  const long long w_at = group * a.weight_gstride;
  for (int c = threadIdx.x; c < 2 * a.width; c += kThreads) acc[c] = 0.0f;
  for (int r = r0; r < r1; ++r) {
    const long long row = (long long)group * a.seq + r;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
    const float mean = kRms ? 0.0f : a.mean[row];
    float s = 0.0f, q = 0.0f;  // layer norm: sums of g and g (x - mean); rms: of x^2 and g x
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      const float w = param_at(a.weight, a.param_dtype, w_at + c, kRms ? 0.0f : 1.0f) + (kRms ? 1.0f : 0.0f);
      const float g = to_f32(dy[c]) * w, d = to_f32(x[c]) - mean;
      s = kRms ? fmaf(d, d, s) : s + g;
      q = fmaf(g, d, q);
    }
    const float2 t = cta_sum2(s, q, sums);
    const float rstd = kRms ? rsqrtf(t.x * inv + a.eps) : a.rstd[row];
    const float mg = kRms ? 0.0f : t.x * inv, mgn = t.y * rstd * inv;
    bool live = true;
    if (!(fabsf(mgn) <= 3.402823466e38f) || !(fabsf(rstd) <= 3.402823466e38f) || !(fabsf(mean) <= 3.402823466e38f)) {
      // not finite: a row without a gradient is left out, any other keeps what it has
      int any = 0;
      for (int c = threadIdx.x; c < a.width; c += kThreads) any |= to_f32(dy[c]) != 0.0f;
      live = __syncthreads_or(any) != 0;
    }
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      float o = a.residual != nullptr ? to_f32((static_cast<const T*>(a.residual) + row * a.residual_stride)[c]) : 0.0f;
      if (live) {
        const float w = param_at(a.weight, a.param_dtype, w_at + c, kRms ? 0.0f : 1.0f) + (kRms ? 1.0f : 0.0f);
        const float y = to_f32(dy[c]), n = (to_f32(x[c]) - mean) * rstd;
        acc[c] = fmaf(y, n, acc[c]);
        acc[a.width + c] += y;
        o = fmaf(rstd, y * w - mg - n * mgn, o);
      }
      from_f32(o, dx[c]);
    }
  }
  __syncthreads();
  float* to = a.partial + (long long)blockIdx.x * 2 * a.width;
  for (int c = threadIdx.x; c < 2 * a.width; c += kThreads) to[c] = acc[c];
}

// The sums of the parts, in order.
__global__ void __launch_bounds__(kThreads) norm_sum_kernel(const float* __restrict__ partial, int parts, int width,
                                                            float* dweight, float* dbias, long long sum_gstride) {
  grid_dep_wait();
  grid_dep_launch();
  const int blocks = (width + kThreads - 1) / kThreads, group = blockIdx.x / blocks;
  const int c = blockIdx.x % blocks * kThreads + threadIdx.x;
  if (c >= width) return;
  const float* p = partial + (long long)group * parts * 2 * width + c;
  float w = 0.0f, b = 0.0f;
  for (int i = 0; i < parts; ++i) {
    w += p[(long long)i * 2 * width];
    b += p[(long long)i * 2 * width + width];
  }
  const long long at = group * sum_gstride + c;
  if (dweight == dbias && dweight != nullptr) {
    dweight[at] = w + b;
    return;
  }
  if (dweight != nullptr) dweight[at] = w;
  if (dbias != nullptr) dbias[at] = b;
}

int norm_bwd_parts(int groups, int seq, int num_sms) {
  const int most = (2 * num_sms + groups - 1) / groups;
  return seq < most ? seq : most;
}

template <typename T, bool kRms>
cudaError_t norm_bwd_run(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  const int parts = norm_bwd_parts(a.groups, a.seq, num_sms);
  if (parts > 0) {
    const size_t smem = (size_t)2 * a.width * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, kRms>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         2 * MI_NORM_MAX_WIDTH * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    e = launch_kernel(norm_bwd_kernel<T, kRms>, dim3(parts * a.groups), dim3(kThreads), smem, s, true, a, parts);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
  return launch_kernel(norm_sum_kernel, dim3((a.width + kThreads - 1) / kThreads * a.groups), dim3(kThreads), 0, s, true,
                       (const float*)a.partial, parts, a.width, a.dweight, a.dbias, a.sum_gstride);
}

}  // namespace

cudaError_t layer_norm_launch(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  const int cap = 8 * num_sms;
  const dim3 grid(a.rows < cap ? a.rows : cap);
  if (a.dtype == MI_F32) return launch_kernel(layer_norm_kernel<float>, grid, dim3(kThreads), 0, s, true, a);
  if (a.dtype == MI_F16) return launch_kernel(layer_norm_kernel<__half>, grid, dim3(kThreads), 0, s, true, a);
  return launch_kernel(layer_norm_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, true, a);
}

size_t norm_bwd_workspace(int groups, int seq, int width, int num_sms) {
  return (size_t)groups * norm_bwd_parts(groups, seq, num_sms) * 2 * width * sizeof(float);
}

cudaError_t norm_bwd_launch(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  if (a.rms) return norm_bwd_run<__nv_bfloat16, true>(a, num_sms, s);
  if (a.dtype == MI_F32) return norm_bwd_run<float, false>(a, num_sms, s);
  if (a.dtype == MI_F16) return norm_bwd_run<__half, false>(a, num_sms, s);
  return norm_bwd_run<__nv_bfloat16, false>(a, num_sms, s);
}

}  // namespace mi
