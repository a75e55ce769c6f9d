// Layer norm, and its form without the mean (rms), in front of the head:
// forward with the residual add, and backward with the column sums that give
// the weight's and the bias's gradient.
//
// Both move every element once and compute about ten operations on it, so
// memory bandwidth bounds them (4 N H b bytes forward and backward with a
// residual, b bytes an element); for few rows the latency of one row does.
#include <math.h>

#include <algorithm>

#include "elem.cuh"
#include "ptx.cuh"

namespace flce {
namespace {

// Column sums of the backward pass are taken by at most this many CTAs, each
// leaving one partial row of H sums (the workspace holds them all).
constexpr int kMaxParts = 304;

struct LnForward {
  const void *x, *residual, *weight, *bias;
  void *y, *sum;
  float *mean, *rstd;
  int64_t ld_x, ld_residual, ld_y, ld_sum, N, H;
  float eps;
  int param_dtype;
};

struct LnBackward {
  const void *grad_y, *x, *weight, *grad_sum;
  const float *mean, *rstd;
  void* grad_x;
  int64_t ld_grad_y, ld_x, ld_grad_sum, ld_grad_x, N, H;
  int param_dtype;
  float2* row_terms;   // [N]: mean(u) * rstd, mean(u * xhat) * rstd
  float *part_w, *part_b;  // [parts][H]
  int parts;
};

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

// A row as the 16-byte vectors that cover it.  Without SHIFTED the row is a whole
// number of them.  With it the row starts `shift` elements into its first one and
// ends anywhere in its last: these two are read and written element by element,
// what is not the row's reading as 0.
template <typename T, bool SHIFTED>
struct Row {
  static constexpr int kN = Vec<T>::kN;
  int shift, length, vectors;
  __device__ __forceinline__ Row(const void* first, int64_t H) {
    length = static_cast<int>(H);
    shift = SHIFTED ? static_cast<int>(reinterpret_cast<uintptr_t>(first) % 16 / sizeof(T)) : 0;
    vectors = (shift + length + kN - 1) / kN;
  }
  __device__ __forceinline__ int column(int j) const { return j * kN - shift; }  // of vector j's first element
  __device__ __forceinline__ bool whole(int j) const {
    return !SHIFTED || (j * kN >= shift && (j + 1) * kN <= shift + length);
  }
  __device__ __forceinline__ bool inside(int c) const { return !SHIFTED || (c >= 0 && c < length); }
  __device__ __forceinline__ uint4 load(const T* row, int j) const {
    if (whole(j)) return *reinterpret_cast<const uint4*>(row + column(j));
    float f[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) f[k] = inside(column(j) + k) ? to_float(row[column(j) + k]) : 0.f;
    return Vec<T>::pack(f);
  }
  __device__ __forceinline__ void store(T* row, int j, const uint4& v) const {
    if (whole(j)) {
      *reinterpret_cast<uint4*>(row + column(j)) = v;
      return;
    }
    float f[kN];
    Vec<T>::unpack(v, f);
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (inside(column(j) + k)) row[column(j) + k] = from_float<T>(f[k]);
  }
  // Weights or biases of vector j's columns (which never change while a kernel runs).
  __device__ __forceinline__ void params(const void* p, int dtype, int j, float* f) const {
    const int c = column(j);
    if (!SHIFTED) {
#pragma unroll
      for (int k = 0; k < kN; k += 4) {
        float4 v;
        if (dtype == FLCE_DTYPE_FP32) {
          v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + k));
        } else {
          const uint2 h = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c + k));
          v = four_floats(make_uint4(h.x, h.y, 0, 0), dtype);
        }
        f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
      }
      return;
    }
    int at[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) at[k] = min(max(c + k, 0), length - 1);
    if (dtype == FLCE_DTYPE_FP32) {
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] = __ldg(static_cast<const float*>(p) + at[k]);
    } else if (dtype == FLCE_DTYPE_BF16) {
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] = to_float(__ldg(static_cast<const __nv_bfloat16*>(p) + at[k]));
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k) f[k] = to_float(__ldg(static_cast<const __half*>(p) + at[k]));
    }
  }
};

// Sum over a row's threads: one warp, or the CTA (`scratch`: 32 numbers that no
// other sum of the kernel uses).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
  v = warp_sum(v);
  if (WARP) return v;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? scratch[lane] : 0.f);
}

// Forward with the row in registers, VPT vectors a thread: a warp (WARP) or a CTA
// takes one row, which is read once; the mean and then the sum of squares about it
// are taken from the registers.
template <typename T, bool RMS, int VPT, bool WARP, bool SHIFTED>
__global__ void __launch_bounds__(WARP ? 256 : 1024) ln_fwd_kernel(const LnForward p) {
  using V = Vec<T>;
  __shared__ float scratch[2][32];
  const int threads = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t n = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (n >= p.N) return;
  const T* x = static_cast<const T*>(p.x) + n * p.ld_x;
  const Row<T, SHIFTED> row(x, p.H);
  uint4 v[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int j = t + k * threads;
    v[k] = j < row.vectors ? row.load(x, j) : make_uint4(0, 0, 0, 0);
  }
  if (p.residual != nullptr) {
    const T* r = static_cast<const T*>(p.residual) + n * p.ld_residual;
    uint4 w[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = t + k * threads;
      w[k] = j < row.vectors ? row.load(r, j) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float a[V::kN], b[V::kN];
      V::unpack(v[k], a);
      V::unpack(w[k], b);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) a[i] += b[i];
      v[k] = V::pack(a);
    }
    if (p.sum != nullptr) {
      T* s = static_cast<T*>(p.sum) + n * p.ld_sum;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (t + k * threads < row.vectors) row.store(s, t + k * threads, v[k]);
    }
  }
  const float over = 1.f / static_cast<float>(row.length);
  float mu = 0.f;
  if (!RMS) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float f[V::kN];
      V::unpack(v[k], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) a += f[i];
    }
    mu = row_sum<WARP>(a, scratch[0]) * over;
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int j = t + k * threads;
    if (RMS || j < row.vectors) {
      const bool all = RMS || row.whole(j);
      float f[V::kN];
      V::unpack(v[k], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) {
        const float d = f[i] - mu;
        if (all || row.inside(row.column(j) + i)) q = fmaf(d, d, q);
      }
    }
  }
  q = row_sum<WARP>(q, scratch[1]) * over;
  const float inv = rsqrtf(q + p.eps);
  T* y = static_cast<T*>(p.y) + n * p.ld_y;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int j = t + k * threads;
    if (j < row.vectors) {
      float f[V::kN];
      V::unpack(v[k], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) f[i] = (f[i] - mu) * inv;
      if (p.weight != nullptr) {
        float w[V::kN];
        row.params(p.weight, p.param_dtype, j, w);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) f[i] *= w[i];
      }
      if (p.bias != nullptr) {
        float b[V::kN];
        row.params(p.bias, p.param_dtype, j, b);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) f[i] += b[i];
      }
      row.store(y, j, V::pack(f));
    }
  }
  if (t == 0) {
    if (p.mean != nullptr) p.mean[n] = mu;
    if (p.rstd != nullptr) p.rstd[n] = inv;
  }
}

// ------------------------------------------------------- any layout, by elements

constexpr int kAnyThreads = 256;

// One CTA a row, element by element, the row read again for each of its three
// uses (mean, sum of squares about it, output): the form for rows that 16-byte
// vectors do not fit.
template <typename T, bool RMS>
__global__ void __launch_bounds__(kAnyThreads) ln_fwd_any_kernel(const LnForward p) {
  __shared__ float2 scratch[32];
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + n * p.ld_x;
    const T* r = p.residual != nullptr ? static_cast<const T*>(p.residual) + n * p.ld_residual : nullptr;
    T* y = static_cast<T*>(p.y) + n * p.ld_y;
    T* s = p.sum != nullptr ? static_cast<T*>(p.sum) + n * p.ld_sum : nullptr;
    const auto at = [&](int64_t h) {
      const float v = to_float(x[h]);
      return r != nullptr ? to_float(from_float<T>(v + to_float(r[h]))) : v;
    };
    float mu = 0.f;
    if (!RMS) {
      float a = 0.f;
      for (int64_t h = threadIdx.x; h < p.H; h += kAnyThreads) a += at(h);
      mu = block_sum2(make_float2(a, 0.f), scratch).x / static_cast<float>(p.H);
    }
    float q = 0.f;
    for (int64_t h = threadIdx.x; h < p.H; h += kAnyThreads) {
      const float d = at(h) - mu;
      q += d * d;
    }
    q = block_sum2(make_float2(q, 0.f), scratch).x / static_cast<float>(p.H);
    const float inv = rsqrtf(q + p.eps);
    for (int64_t h = threadIdx.x; h < p.H; h += kAnyThreads) {
      const float v = at(h);
      float o = (v - mu) * inv;
      if (p.weight != nullptr) o *= load_elem(p.weight, p.param_dtype, h);
      if (p.bias != nullptr) o += load_elem(p.bias, p.param_dtype, h);
      if (s != nullptr) s[h] = from_float<T>(v);
      y[h] = from_float<T>(o);
    }
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[n] = mu;
      if (p.rstd != nullptr) p.rstd[n] = inv;
    }
  }
}

// The two row means of the backward pass, one CTA a row.
template <typename T, bool RMS>
__global__ void __launch_bounds__(kAnyThreads) ln_bwd_rows_any_kernel(const LnBackward p) {
  __shared__ float2 scratch[32];
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + n * p.ld_x;
    const T* g = static_cast<const T*>(p.grad_y) + n * p.ld_grad_y;
    const float mu = RMS ? 0.f : p.mean[n], inv = p.rstd[n];
    float2 a = make_float2(0.f, 0.f);
    for (int64_t h = threadIdx.x; h < p.H; h += kAnyThreads) {
      float u = to_float(g[h]);
      if (p.weight != nullptr) u *= load_elem(p.weight, p.param_dtype, h);
      a.x += u;
      a.y += u * ((to_float(x[h]) - mu) * inv);
    }
    a = block_sum2(a, scratch);
    if (threadIdx.x == 0) p.row_terms[n] = make_float2(RMS ? 0.f : a.x / p.H, a.y / p.H);
  }
}

// grad_x and the column sums, 64 columns by 4 rows a CTA at a time: CTA
// (c, s) takes columns 64 c.. and the s-th of gridDim.y ranges of rows.
template <typename T, bool RMS>
__global__ void __launch_bounds__(kAnyThreads) ln_bwd_cols_any_kernel(const LnBackward p) {
  __shared__ float2 scratch[4][64];
  const int col = threadIdx.x & 63, lane = threadIdx.x >> 6;
  const int64_t h = static_cast<int64_t>(blockIdx.x) * 64 + col;
  const int64_t per = (p.N + gridDim.y - 1) / gridDim.y;
  const int64_t n0 = per * blockIdx.y, n1 = min(n0 + per, p.N);
  float sw = 0.f, sb = 0.f;
  if (h < p.H) {
    const float w = p.weight != nullptr ? load_elem(p.weight, p.param_dtype, h) : 1.f;
    for (int64_t n = n0 + lane; n < n1; n += 4) {
      const float mu = RMS ? 0.f : p.mean[n], inv = p.rstd[n];
      const float g = to_float(static_cast<const T*>(p.grad_y)[n * p.ld_grad_y + h]);
      const float xhat = (to_float(static_cast<const T*>(p.x)[n * p.ld_x + h]) - mu) * inv;
      sw += g * xhat;
      sb += g;
      if (p.grad_x != nullptr) {
        const float2 t = p.row_terms[n];
        float o = (g * w - t.x - xhat * t.y) * inv;
        if (p.grad_sum != nullptr) o += to_float(static_cast<const T*>(p.grad_sum)[n * p.ld_grad_sum + h]);
        static_cast<T*>(p.grad_x)[n * p.ld_grad_x + h] = from_float<T>(o);
      }
    }
  }
  scratch[lane][col] = make_float2(sw, sb);
  __syncthreads();
  if (lane == 0 && h < p.H) {
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a.x += scratch[k][col].x;
      a.y += scratch[k][col].y;
    }
    if (p.part_w != nullptr) p.part_w[static_cast<int64_t>(blockIdx.y) * p.H + h] = a.x;
    if (p.part_b != nullptr) p.part_b[static_cast<int64_t>(blockIdx.y) * p.H + h] = a.y;
  }
}

// Adds the partial rows of column sums in a fixed order: 32 columns by 32
// lanes a CTA, blockIdx.y 0 the weight's and 1 the bias's.
__global__ void __launch_bounds__(1024)
    ln_reduce_kernel(const float* part_w, const float* part_b, int parts, int64_t H, float* grad_weight,
                     float* grad_bias, int accumulate) {
  __shared__ float scratch[32][33];
  grid_dependency_wait();
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? grad_weight : grad_bias;
  if (out == nullptr) return;
  const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int64_t h = static_cast<int64_t>(blockIdx.x) * 32 + col;
  float a = 0.f;
  if (h < H)
    for (int k = lane; k < parts; k += 32) a += part[static_cast<int64_t>(k) * H + h];
  scratch[lane][col] = a;
  __syncthreads();
  a = warp_sum(scratch[col][lane]);  // lane `col` of warp `lane`: partial `col` of column `lane`
  const int64_t ho = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  if (col == 0 && ho < H) out[ho] = accumulate ? out[ho] + a : a;
}

// ------------------------------------------------------------------ launches

// How a call's matrices lie to 16-byte vectors.
enum Fit {
  kFitNot,      // rows of different matrices start at different places of a vector
  kFitShifted,  // at the same place, row by row
  kFitWhole     // at a vector's start, with a whole number of vectors
};

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
  return whole ? kFitWhole : kFitShifted;
}

// Most vectors of a row that the register forms take (eight for each of 1024 threads).
constexpr int64_t kMaxRowVectors = 8192;

template <typename T, bool RMS, bool SHIFTED>
void forward_rows(const LnForward& p, int64_t vectors, cudaStream_t s) {
  const unsigned int rows = static_cast<unsigned int>(p.N), warps = 4;
  const unsigned int grid = (rows + warps - 1) / warps;
  if (vectors <= 32) {
    ln_fwd_kernel<T, RMS, 1, true, SHIFTED><<<grid, 32 * warps, 0, s>>>(p);
  } else if (vectors <= 64) {
    ln_fwd_kernel<T, RMS, 2, true, SHIFTED><<<grid, 32 * warps, 0, s>>>(p);
  } else if (vectors <= 128) {
    ln_fwd_kernel<T, RMS, 4, true, SHIFTED><<<grid, 32 * warps, 0, s>>>(p);
  } else if (vectors <= 4096) {
    ln_fwd_kernel<T, RMS, 4, false, SHIFTED><<<rows, static_cast<unsigned int>(div_up(vectors, 128) * 32), 0, s>>>(p);
  } else {
    ln_fwd_kernel<T, RMS, 8, false, SHIFTED><<<rows, 1024, 0, s>>>(p);
  }
}

template <typename T, bool RMS>
cudaError_t forward(const LnForward& p, cudaStream_t s) {
  const Fit fit = fit_of<T>(p.N, p.H, p.weight, p.bias, p.param_dtype, Matrix{p.x, p.ld_x},
                            Matrix{p.residual, p.ld_residual}, Matrix{p.y, p.ld_y}, Matrix{p.sum, p.ld_sum});
  const int64_t vectors = fit == kFitWhole ? p.H / Vec<T>::kN : div_up(p.H + Vec<T>::kN - 1, Vec<T>::kN);
  prof_begin(s, FLCE_KERNEL_LN_FWD);
  if (fit == kFitNot || vectors > kMaxRowVectors)
    ln_fwd_any_kernel<T, RMS>
        <<<static_cast<int>(std::min<int64_t>(p.N, int64_t(8) * device_sm_count())), kAnyThreads, 0, s>>>(p);
  else if (fit == kFitWhole)
    forward_rows<T, RMS, false>(p, vectors, s);
  else
    forward_rows<T, RMS, true>(p, vectors, s);
  const cudaError_t e = cudaGetLastError();
  prof_end(s);
  return e;
}

cudaError_t reduce_columns(const LnBackward& p, float* grad_weight, float* grad_bias, int accumulate,
                           cudaStream_t s) {
  if (grad_weight == nullptr && grad_bias == nullptr) return cudaSuccess;
  prof_begin(s, FLCE_KERNEL_LN_REDUCE);
  ln_reduce_kernel<<<dim3(static_cast<unsigned>(div_up(p.H, 32)), 2), 1024, 0, s>>>(
      p.part_w, p.part_b, p.parts, p.H, grad_weight, grad_bias, accumulate);
  const cudaError_t e = cudaGetLastError();
  prof_end(s);
  return e;
}

template <typename T, bool RMS>
cudaError_t backward(LnBackward p, float* grad_weight, float* grad_bias, int accumulate, cudaStream_t s) {
  p.parts = 0;
  if (p.N > 0) {
    const int sms = device_sm_count();
    if (p.grad_x != nullptr) {
      prof_begin(s, FLCE_KERNEL_LN_BWD);
      ln_bwd_rows_any_kernel<T, RMS>
          <<<static_cast<int>(std::min<int64_t>(p.N, int64_t(8) * sms)), kAnyThreads, 0, s>>>(p);
      const cudaError_t e = cudaGetLastError();
      prof_end(s);
      if (e != cudaSuccess) return e;
    }
    const int64_t strips = div_up(p.H, 64);
    p.parts = static_cast<int>(std::min<int64_t>({div_up(int64_t(8) * sms, strips), div_up(p.N, 4), kMaxParts}));
    prof_begin(s, FLCE_KERNEL_LN_BWD);
    ln_bwd_cols_any_kernel<T, RMS><<<dim3(static_cast<unsigned>(strips), p.parts), kAnyThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    prof_end(s);
    if (e != cudaSuccess) return e;
  }
  return reduce_columns(p, grad_weight, grad_bias, accumulate, s);
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

struct LnLayout {
  size_t row_terms, part_w, part_b, total;
};

LnLayout ln_layout(int64_t N, int64_t H) {
  LnLayout L;
  const size_t part = align_up(static_cast<size_t>(std::min<int64_t>(std::max<int64_t>(N, 1), kMaxParts)) * H * 4, 256);
  L.row_terms = 0;
  L.part_w = align_up(static_cast<size_t>(N) * sizeof(float2), 256);
  L.part_b = L.part_w + part;
  L.total = L.part_b + part;
  return L;
}

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

using namespace flce;

extern "C" {

flce_status_t ln_fwd(int kind, int dtype, const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                     const void* weight, const void* bias, int param_dtype, int64_t N, int64_t H, float eps,
                     void* y, int64_t ld_y, void* sum, int64_t ld_sum, float* mean, float* rstd,
                     flce_stream_t stream_) {
  if (kind != FLCE_NORM_LAYER && kind != FLCE_NORM_RMS) return FLCE_ERR_INVALID_ARG;
  if (!float_dtype(dtype) || !float_dtype(param_dtype)) return FLCE_ERR_UNSUPPORTED;
  if (!sizes_ok(N, H) || !(eps >= 0.f)) return FLCE_ERR_INVALID_ARG;
  if (ld_x < 0 || ld_x > kMaxLd || ld_y < H || ld_y > kMaxLd) return FLCE_ERR_INVALID_ARG;
  if (residual != nullptr && (ld_residual < 0 || ld_residual > kMaxLd)) return FLCE_ERR_INVALID_ARG;
  if (sum != nullptr && (residual == nullptr || ld_sum < H || ld_sum > kMaxLd)) return FLCE_ERR_INVALID_ARG;
  if (mean != nullptr && kind == FLCE_NORM_RMS) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (x == nullptr || y == nullptr)) return FLCE_ERR_INVALID_ARG;
  const size_t esz = elem_size(dtype), psz = elem_size(param_dtype);
  if (!aligned_to(x, esz) || !aligned_to(residual, esz) || !aligned_to(y, esz) || !aligned_to(sum, esz) ||
      !aligned_to(weight, psz) || !aligned_to(bias, psz) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return FLCE_ERR_MISALIGNED;
  if (clashes(y, ld_y, x, ld_x, N, H, esz) || clashes(y, ld_y, residual, ld_residual, N, H, esz) ||
      clashes(sum, ld_sum, x, ld_x, N, H, esz) || clashes(sum, ld_sum, residual, ld_residual, N, H, esz) ||
      overlap(y, ld_y, sum, ld_sum, N, H, esz))
    return FLCE_ERR_INVALID_ARG;
  if (N == 0) return FLCE_OK;
  LnForward p = {x, residual, weight, bias, y, sum, mean, rstd, ld_x, ld_residual, ld_y, ld_sum, N, H, eps, param_dtype};
  return LN_BY_TYPE(forward, p, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

size_t ln_workspace_size(int64_t N, int64_t H) { return sizes_ok(N, H) ? ln_layout(N, H).total : 0; }

flce_status_t ln_bwd(int kind, int dtype, const void* grad_y, int64_t ld_grad_y, const void* x, int64_t ld_x,
                     const void* weight, int param_dtype, const float* mean, const float* rstd,
                     const void* grad_sum, int64_t ld_grad_sum, int64_t N, int64_t H, void* grad_x,
                     int64_t ld_grad_x, float* grad_weight, float* grad_bias, int accumulate, void* workspace,
                     size_t workspace_bytes, flce_stream_t stream_) {
  if (kind != FLCE_NORM_LAYER && kind != FLCE_NORM_RMS) return FLCE_ERR_INVALID_ARG;
  if (!float_dtype(dtype) || !float_dtype(param_dtype)) return FLCE_ERR_UNSUPPORTED;
  if (!sizes_ok(N, H) || (accumulate != 0 && accumulate != 1)) return FLCE_ERR_INVALID_ARG;
  if (ld_grad_y < 0 || ld_grad_y > kMaxLd || ld_x < 0 || ld_x > kMaxLd) return FLCE_ERR_INVALID_ARG;
  if (grad_sum != nullptr && (ld_grad_sum < 0 || ld_grad_sum > kMaxLd)) return FLCE_ERR_INVALID_ARG;
  if (grad_x != nullptr && (ld_grad_x < H || ld_grad_x > kMaxLd)) return FLCE_ERR_INVALID_ARG;
  if (grad_sum != nullptr && grad_x == nullptr) return FLCE_ERR_INVALID_ARG;
  if (mean != nullptr && kind == FLCE_NORM_RMS) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && (grad_y == nullptr || x == nullptr || rstd == nullptr || (kind == FLCE_NORM_LAYER && mean == nullptr)))
    return FLCE_ERR_INVALID_ARG;
  const size_t esz = elem_size(dtype), psz = elem_size(param_dtype);
  if (!aligned_to(grad_y, esz) || !aligned_to(x, esz) || !aligned_to(grad_sum, esz) || !aligned_to(grad_x, esz) ||
      !aligned_to(weight, psz) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(grad_weight, 4) ||
      !aligned_to(grad_bias, 4))
    return FLCE_ERR_MISALIGNED;
  if (clashes(grad_x, ld_grad_x, grad_y, ld_grad_y, N, H, esz) || clashes(grad_x, ld_grad_x, x, ld_x, N, H, esz) ||
      clashes(grad_x, ld_grad_x, grad_sum, ld_grad_sum, N, H, esz))
    return FLCE_ERR_INVALID_ARG;
  if (grad_x == nullptr && grad_weight == nullptr && grad_bias == nullptr) return FLCE_OK;
  const LnLayout L = ln_layout(N, H);
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < L.total) return FLCE_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LnBackward p = {grad_y, x, weight, grad_sum, mean, rstd, grad_x, ld_grad_y, ld_x, ld_grad_sum, ld_grad_x, N, H,
                  param_dtype, reinterpret_cast<float2*>(ws + L.row_terms),
                  grad_weight != nullptr ? reinterpret_cast<float*>(ws + L.part_w) : nullptr,
                  grad_bias != nullptr ? reinterpret_cast<float*>(ws + L.part_b) : nullptr, 0};
  return LN_BY_TYPE(backward, p, grad_weight, grad_bias, accumulate, reinterpret_cast<cudaStream_t>(stream_)) ==
                 cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

}  // extern "C"
