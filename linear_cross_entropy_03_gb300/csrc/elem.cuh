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

// Four elements from i on, which lie on a boundary of four; read or written once
// (streamed: first to leave the caches).  Loading and converting are apart, so
// that several loads are under way before the first is waited for.
__device__ __forceinline__ uint4 load_four_bits(const void* p, int dtype, int64_t i) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if (dtype == FLCE_DTYPE_FP32) {
    r = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i));
  } else {
    const uint2 h = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    r.x = h.x;
    r.y = h.y;
  }
  return r;
}
__device__ __forceinline__ float4 four_floats(const uint4& r, int dtype) {
  if (dtype == FLCE_DTYPE_FP32)
    return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
  if (dtype == FLCE_DTYPE_BF16)
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
  const float2 a = __half22float2(reinterpret_cast<const __half2&>(r.x));
  const float2 b = __half22float2(reinterpret_cast<const __half2&>(r.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_four(void* p, int dtype, int64_t i, const float4& v) {
  if (dtype == FLCE_DTYPE_FP32) {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + i), v);
    return;
  }
  uint2 r;
  if (dtype == FLCE_DTYPE_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    r = make_uint2(reinterpret_cast<const uint32_t&>(a), reinterpret_cast<const uint32_t&>(b));
  } else {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    r = make_uint2(reinterpret_cast<const uint32_t&>(a), reinterpret_cast<const uint32_t&>(b));
  }
  __stcs(reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i), r);
}

// Two fp32 operations in one instruction.
struct Pair {
  uint64_t v;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ Pair pair(float both) { return pair(both, both); }
__device__ __forceinline__ float2 unpair(Pair a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair fma_pair(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// load_four_bits' four elements as two pairs.
__device__ __forceinline__ void four_pairs(const uint4& r, int dtype, Pair* to) {
  const float4 f = four_floats(r, dtype);
  to[0] = pair(f.x, f.y);
  to[1] = pair(f.z, f.w);
}

inline bool float_dtype(int dtype) {
  return dtype == FLCE_DTYPE_BF16 || dtype == FLCE_DTYPE_FP16 || dtype == FLCE_DTYPE_FP32;
}
inline size_t elem_size(int dtype) { return dtype == FLCE_DTYPE_FP32 ? 4 : 2; }
// Whether p is a multiple of `a`, a power of 2.
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Launches a kernel that may start while its predecessor on the stream still
// runs, up to its griddepcontrol.wait; with `smem` bytes of dynamic shared memory.
template <typename... P, typename... A>
cudaError_t launch_after_with(size_t smem, void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  return launch_after_with(0, kernel, grid, block, s, args...);
}

}  // namespace flce
