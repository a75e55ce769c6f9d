// What the layer norm's forward and backward pass share: rows as 16-byte vectors,
// sums over a row's threads, and the checks of their arguments.
#pragma once

#include <algorithm>

#include "elem.cuh"
#include "ptx.cuh"

namespace flce {
namespace {

// ------------------------------------------------------- rows by 16-byte vectors

// The elements of 16 bytes.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(reinterpret_cast<const __half2&>(w[k]));
      f[2 * k] = v.x, f[2 * k + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
      w[k] = reinterpret_cast<const uint32_t&>(h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// OUT words from a 4-byte boundary on, by 16-byte loads from the boundary of 16 before
// it (of memory that never changes while a kernel runs).
template <int OUT>
__device__ __forceinline__ void words_at(uintptr_t from, uint32_t* out) {
  constexpr int kLoads = (OUT + 6) / 4;
  uint32_t w[kLoads * 4];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(from & ~uintptr_t(15)) + k);
    w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
  }
#pragma unroll
  for (int k = 0; k < OUT + 1; ++k) w[k] = from & 8 ? w[k + 2] : w[k];
#pragma unroll
  for (int k = 0; k < OUT; ++k) out[k] = from & 4 ? w[k + 1] : w[k];
}

// A row as 16-byte vectors.  Without SHIFTED it is a whole number of them.  With it,
// vectors start at the boundaries of 16 bytes inside the row, `before` elements (at
// least kMargin) after its start, and end at least kMargin before its end; what lies
// before and after, at most 30 elements, goes one by one to the row's first threads.
// The margins keep the reads of a vector's weights (below) inside their array.
template <typename T, bool SHIFTED>
struct Row {
  static constexpr int kN = Vec<T>::kN;
  static constexpr int kMargin = kN == 8 ? 8 : 12;
  int before, vectors, length;
  __device__ __forceinline__ Row(const void* first, int64_t H) {
    length = static_cast<int>(H);
    before = 0;
    vectors = length / kN;
    if (SHIFTED) {
      before = kMargin + (kN - (static_cast<int>(reinterpret_cast<uintptr_t>(first) / sizeof(T)) + kMargin) % kN) % kN;
      vectors = (length - before - kMargin) / kN;
    }
  }
  __device__ __forceinline__ int column(int j) const { return before + j * kN; }  // of vector j's first element
  // The column that thread t of the row has beside its vectors, or -1.
  __device__ __forceinline__ int extra(int t) const {
    if (!SHIFTED) return -1;
    const int c = t < before ? t : t + vectors * kN;
    return c < length ? c : -1;
  }
  __device__ __forceinline__ uint4 load(const T* row, int j) const {
    return *reinterpret_cast<const uint4*>(row + column(j));
  }
  __device__ __forceinline__ void store(T* row, int j, const uint4& v) const {
    *reinterpret_cast<uint4*>(row + column(j)) = v;
  }
  // Weights or biases of vector j's columns (which never change while a kernel runs).
  __device__ __forceinline__ void params(const void* p, int dtype, int j, float* f) const {
    const int c = column(j);
    if constexpr (!SHIFTED) {
#pragma unroll
      for (int q = 0; q < kN / 4; ++q) {
        const int k = 4 * q;
        float4 v;
        if (dtype == FLCE_DTYPE_FP32) {
          v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + k));
        } else {
          const uint2 h = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c + k));
          v = four_floats(make_uint4(h.x, h.y, 0, 0), dtype);
        }
        f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
      }
    } else if (dtype == FLCE_DTYPE_FP32) {
      uint32_t w[kN];
      words_at<kN>(reinterpret_cast<uintptr_t>(static_cast<const float*>(p) + c), w);
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] = __uint_as_float(w[k]);
    } else {
      const uintptr_t from = reinterpret_cast<uintptr_t>(static_cast<const uint16_t*>(p) + c);
      const unsigned int pick = from & 2 ? 0x5432 : 0x3210;
      uint32_t w[kN / 2 + 1];
      words_at<kN / 2 + 1>(from & ~uintptr_t(3), w);
#pragma unroll
      for (int k = 0; k < kN / 4; ++k) {
        const float4 v = four_floats(make_uint4(__byte_perm(w[2 * k], w[2 * k + 1], pick),
                                                __byte_perm(w[2 * k + 1], w[2 * k + 2], pick), 0, 0), dtype);
        f[4 * k] = v.x, f[4 * k + 1] = v.y, f[4 * k + 2] = v.z, f[4 * k + 3] = v.w;
      }
    }
  }
};

// ------------------------------------------------------- any layout, by elements

constexpr int kAnyThreads = 256;

// Terms that a thread adds up before it adds their sum to the others': chains of fp32
// additions as long as a row or a range of rows lose bits (16384 equal terms 1e-4 of their sum).
constexpr int64_t kBatch = 64;

// Sum over the CTA's threads (a multiple of 32, at most 1024), to all of them.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* scratch) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();  // the scratch of an earlier sum has been read
  if (lane == 0) scratch[warp] = v;
  __syncthreads();
  v = lane < warps ? scratch[lane] : make_float2(0.f, 0.f);
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  return v;
}

// Sums of at(h).x and at(h).y over the columns of this thread of a CTA of kAnyThreads.
template <typename F>
__device__ __forceinline__ float2 thread_sum2(int64_t H, F at) {
  float2 sum = make_float2(0.f, 0.f);
  for (int64_t h = threadIdx.x; h < H;) {
    const int64_t end = min(h + kBatch * kAnyThreads, H);
    float2 batch = make_float2(0.f, 0.f);
    for (; h < end; h += kAnyThreads) {
      const float2 v = at(h);
      batch.x += v.x;
      batch.y += v.y;
    }
    sum.x += batch.x;
    sum.y += batch.y;
  }
  return sum;
}

// ------------------------------------------------------------------ launches

// How a call's matrices lie to 16-byte vectors.
enum Fit {
  kFitNot,      // rows of different matrices start at different places of a vector
  kFitShifted,  // at the same place, row by row
  kFitWhole     // at a vector's start, with a whole number of vectors
};

constexpr int64_t kMinShifted = 64;  // columns: both margins and a few vectors

struct Matrix {
  const void* p;
  int64_t ld;
};

template <typename T, typename... M>
Fit fit_of(int64_t N, int64_t H, const void* weight, const void* bias, int param_dtype, M... matrices) {
  const Matrix all[] = {matrices...};
  const size_t params = 4 * elem_size(param_dtype);  // parameters are read by fours
  bool whole = H % Vec<T>::kN == 0 && aligned_to(weight, params) && aligned_to(bias, params);
  const uintptr_t start = reinterpret_cast<uintptr_t>(all[0].p) % 16;
  const uintptr_t step = N > 1 ? static_cast<uintptr_t>(all[0].ld) * sizeof(T) % 16 : 0;
  for (const Matrix& m : all) {
    if (m.p == nullptr) continue;
    const uintptr_t s = reinterpret_cast<uintptr_t>(m.p) % 16;
    const uintptr_t d = N > 1 ? static_cast<uintptr_t>(m.ld) * sizeof(T) % 16 : 0;
    if (s != start || d != step) return kFitNot;
    whole = whole && s == 0 && d == 0;
  }
  return whole ? kFitWhole : H >= kMinShifted ? kFitShifted : kFitNot;
}

// ------------------------------------------------------------------- checks

// Whether two matrices of N rows of H elements share memory.  Rows of one
// pitch that lie side by side (columns of one wider matrix) do not.
bool overlap(const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t N, int64_t H, size_t esz) {
  if (a == nullptr || b == nullptr || N == 0) return false;
  const int64_t pa = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a));
  const int64_t pb = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b));
  const int64_t e = static_cast<int64_t>(esz);
  const int64_t bytes_a = ((N - 1) * ld_a + H) * e, bytes_b = ((N - 1) * ld_b + H) * e;
  if (pa >= pb + bytes_b || pb >= pa + bytes_a) return false;
  if (ld_a == ld_b && ld_a > 0 && (pa - pb) % e == 0) {
    int64_t d = (pa - pb) / e % ld_a;
    if (d < 0) d += ld_a;
    if (d >= H && d <= ld_a - H) return false;
  }
  return true;
}

// An output may be an input itself, and nothing in between.
bool clashes(const void* out, int64_t ld_out, const void* in, int64_t ld_in, int64_t N, int64_t H, size_t esz) {
  if (out == in && (ld_out == ld_in || N <= 1)) return false;
  return overlap(out, ld_out, in, ld_in, N, H, esz);
}

bool sizes_ok(int64_t N, int64_t H) {
  return N >= 0 && N < (int64_t(1) << 31) && H >= 1 && H < (int64_t(1) << 24);
}

constexpr int64_t kMaxLd = int64_t(1) << 29;  // N rows of it stay below 2^62 bytes

#define LN_BY_TYPE(fn, ...)                                                                               \
  (kind == FLCE_NORM_RMS                                                                                  \
       ? (dtype == FLCE_DTYPE_BF16   ? fn<__nv_bfloat16, true>(__VA_ARGS__)                               \
          : dtype == FLCE_DTYPE_FP16 ? fn<__half, true>(__VA_ARGS__)                                      \
                                     : fn<float, true>(__VA_ARGS__))                                      \
       : (dtype == FLCE_DTYPE_BF16   ? fn<__nv_bfloat16, false>(__VA_ARGS__)                              \
          : dtype == FLCE_DTYPE_FP16 ? fn<__half, false>(__VA_ARGS__)                                     \
                                     : fn<float, false>(__VA_ARGS__)))

}  // namespace
}  // namespace flce
