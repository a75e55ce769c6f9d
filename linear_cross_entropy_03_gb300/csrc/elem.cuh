// Elements of the three floating types the row and optimiser kernels take
// (bf16, fp16, fp32), and the checks their entry points share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "flce_internal.h"

namespace flce {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Element i of an array whose type is known at run time only.
__device__ __forceinline__ float load_elem(const void* p, int dtype, int64_t i) {
  if (dtype == FLCE_DTYPE_FP32) return static_cast<const float*>(p)[i];
  if (dtype == FLCE_DTYPE_BF16) return to_float(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, int dtype, int64_t i, float v) {
  if (dtype == FLCE_DTYPE_FP32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == FLCE_DTYPE_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = from_float<__nv_bfloat16>(v);
  else
    static_cast<__half*>(p)[i] = from_float<__half>(v);
}

inline bool float_dtype(int dtype) {
  return dtype == FLCE_DTYPE_BF16 || dtype == FLCE_DTYPE_FP16 || dtype == FLCE_DTYPE_FP32;
}
inline size_t elem_size(int dtype) { return dtype == FLCE_DTYPE_FP32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace flce
