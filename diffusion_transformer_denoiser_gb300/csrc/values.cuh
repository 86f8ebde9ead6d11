// Elements of the types that the norms and the clipping take (mi_dtype): in fp32, and back.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/mi_block.h"
#include "ptx.cuh"

namespace mi {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two 16-bit values in a word as fp32, and back (rounded once).
template <typename T> __device__ __forceinline__ f32x2_t unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return f2_pack(t.x, t.y);
  } else {
    return f2_pack(bf16_lo(w), bf16_hi(w));
  }
}
template <typename T> __device__ __forceinline__ uint32_t pack2(f32x2_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// Element i of an array of the given type; p null: `none`.
__device__ __forceinline__ float value_at(const void* p, int dtype, long long i, float none) {
  if (p == nullptr) return none;
  if (dtype == MI_F32) return static_cast<const float*>(p)[i];
  if (dtype == MI_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

}  // namespace mi
