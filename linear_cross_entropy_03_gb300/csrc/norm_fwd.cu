// Layer norm, and its form without the mean (rms), in front of the head: the
// forward pass, with the residual add.
//
// Every element is moved once, with about ten operations on it: memory bandwidth
// bounds it (2 N H b bytes, 4 N H b with a residual, b bytes an element); for few
// rows the latency of one row does.
#include <math.h>

#include "norm.cuh"

namespace flce {
namespace {

struct LnForward {
  const void *x, *residual, *weight, *bias;
  void *y, *sum;
  float *mean, *rstd;
  int64_t ld_x, ld_residual, ld_y, ld_sum, N, H;
  float eps;
  int param_dtype;
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

// (f - mu) inv weight + bias, for a vector of the row and for one element.
template <typename ROW>
__device__ __forceinline__ void finish_vector(const LnForward& p, const ROW& row, int j, float* f, float mu,
                                              float inv) {
#pragma unroll
  for (int e = 0; e < ROW::kN; ++e) f[e] = (f[e] - mu) * inv;
  if (p.weight != nullptr) {
    float w[ROW::kN];
    row.params(p.weight, p.param_dtype, j, w);
#pragma unroll
    for (int e = 0; e < ROW::kN; ++e) f[e] *= w[e];
  }
  if (p.bias != nullptr) {
    float b[ROW::kN];
    row.params(p.bias, p.param_dtype, j, b);
#pragma unroll
    for (int e = 0; e < ROW::kN; ++e) f[e] += b[e];
  }
}
__device__ __forceinline__ float finish_one(const LnForward& p, int c, float f, float mu, float inv) {
  f = (f - mu) * inv;
  if (p.weight != nullptr) f *= load_elem(p.weight, p.param_dtype, c);
  if (p.bias != nullptr) f += load_elem(p.bias, p.param_dtype, c);
  return f;
}

// Forward with the row in registers, VPT vectors a thread: a warp (WARP) takes ROWS
// rows, or a CTA one.  A row is read once; the mean and then the sum of squares about
// it are taken from the registers.  Memory bounds it: bf16 [16384, 4096] with residual
// takes 82 us (6.6 TB/s), fp32 [8191, 2048] 25 us (5.4 TB/s; a plain copy 27 us).  48
// registers a thread let 40 warps have their rows under way on an SM: bf16 [16384,
// 4096] without residual took 51.3 us with 64, 48.2 so, and 55.3 with 32, where some
// are spilled.
template <typename T, bool RMS, int VPT, int ROWS, bool WARP, bool SHIFTED>
__global__ void __maxnreg__(VPT == 8 ? 64 : 48) ln_fwd_kernel(const LnForward p) {
  using V = Vec<T>;
  __shared__ float scratch[2][32];
  const int threads = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first =
      WARP ? (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * ROWS : blockIdx.x;
  const int rows = static_cast<int>(min(p.N - first, static_cast<int64_t>(ROWS)));
  if (rows <= 0) return;
  uint4 v[ROWS][VPT];
  float extra[ROWS];  // SHIFTED: the element beside the vectors
  const auto load = [&](const void* m, int64_t ld, int i, uint4* to, float* one) {
    const T* from = static_cast<const T*>(m) + (first + i) * ld;
    const Row<T, SHIFTED> row(from, p.H);
    const bool there = i < rows;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = t + k * threads;
      to[k] = there && j < row.vectors ? row.load(from, j) : make_uint4(0, 0, 0, 0);
    }
    const int c = row.extra(t);
    *one = there && c >= 0 ? to_float(from[c]) : 0.f;
  };
#pragma unroll
  for (int i = 0; i < ROWS; ++i) load(p.x, p.ld_x, i, v[i], &extra[i]);
  if (p.residual != nullptr) {
    uint4 w[ROWS][VPT];
    float one[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) load(p.residual, p.ld_residual, i, w[i], &one[i]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float a[V::kN], b[V::kN];
        V::unpack(v[i][k], a);
        V::unpack(w[i][k], b);
#pragma unroll
        for (int e = 0; e < V::kN; ++e) a[e] += b[e];
        v[i][k] = V::pack(a);
      }
      extra[i] = to_float(from_float<T>(extra[i] + one[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (i >= rows) return;
    const int64_t n = first + i;
    T* y = static_cast<T*>(p.y) + n * p.ld_y;
    const Row<T, SHIFTED> row(y, p.H);
    const int c = row.extra(t);
    if (p.sum != nullptr) {
      T* s = static_cast<T*>(p.sum) + n * p.ld_sum;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (t + k * threads < row.vectors) row.store(s, t + k * threads, v[i][k]);
      if (c >= 0) s[c] = from_float<T>(extra[i]);
    }
    const float over = 1.f / static_cast<float>(row.length);
    float mu = 0.f;
    if (!RMS) {
      float a = extra[i];
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float f[V::kN];
        V::unpack(v[i][k], f);
#pragma unroll
        for (int e = 0; e < V::kN; ++e) a += f[e];
      }
      mu = row_sum<WARP>(a, scratch[0]) * over;
    }
    float q = c >= 0 ? (extra[i] - mu) * (extra[i] - mu) : 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (RMS || t + k * threads < row.vectors) {
        float f[V::kN];
        V::unpack(v[i][k], f);
#pragma unroll
        for (int e = 0; e < V::kN; ++e) {
          const float d = f[e] - mu;
          q = fmaf(d, d, q);
        }
      }
    }
    q = row_sum<WARP>(q, scratch[1]) * over;
    const float inv = rsqrtf(q + p.eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = t + k * threads;
      if (j < row.vectors) {
        float f[V::kN];
        V::unpack(v[i][k], f);
        finish_vector(p, row, j, f, mu, inv);
        row.store(y, j, V::pack(f));
      }
    }
    if (c >= 0) y[c] = from_float<T>(finish_one(p, c, extra[i], mu, inv));
    if (t == 0) {
      if (p.mean != nullptr) p.mean[n] = mu;
      if (p.rstd != nullptr) p.rstd[n] = inv;
    }
  }
}

// ------------------------------------------------------- any layout, by elements

// One CTA a row, element by element, the row read again for each of its three
// uses (mean, sum of squares about it, output): the form for rows that 16-byte
// vectors do not fit.  Its loads bound it, on short rows the CTA that one takes: fp16
// [8191, 2047] at different places of a vector takes 38 us (floor 10), bf16 [65536, 33]
// 89 (1), bf16 [512, 131072] 398 (40).
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
      const float2 a = thread_sum2(p.H, [&](int64_t h) { return make_float2(at(h), 0.f); });
      mu = block_sum2(a, scratch).x / static_cast<float>(p.H);
    }
    const float2 squares = thread_sum2(p.H, [&](int64_t h) {
      const float d = at(h) - mu;
      return make_float2(d * d, 0.f);
    });
    const float q = block_sum2(squares, scratch).x / static_cast<float>(p.H);
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

// ------------------------------------------------------------------ launches

// Most vectors of a row that the register forms take (eight for each of 1024 threads).
constexpr int64_t kMaxRowVectors = 8192;

template <typename T, bool RMS, bool SHIFTED>
void forward_rows(const LnForward& p, int64_t vectors, cudaStream_t s) {
  constexpr int kWarps = 4;
  // several short rows to a warp once every SM has all the warps it holds (bf16 [65536, 256] 18.5 -> 17.5 us; below,
  // the rows are needed to fill the SMs)
  const int rows = p.N >= int64_t(64) * device_sm_count() ? (vectors <= 32 ? 4 : vectors <= 64 ? 2 : 1) : 1;
  const unsigned int grid = static_cast<unsigned int>(div_up(p.N, kWarps * rows));
  if (vectors <= 32 && rows == 4) {
    ln_fwd_kernel<T, RMS, 1, 4, true, SHIFTED><<<grid, 32 * kWarps, 0, s>>>(p);
  } else if (vectors <= 32) {
    ln_fwd_kernel<T, RMS, 1, 1, true, SHIFTED><<<grid, 32 * kWarps, 0, s>>>(p);
  } else if (vectors <= 64 && rows == 2) {
    ln_fwd_kernel<T, RMS, 2, 2, true, SHIFTED><<<grid, 32 * kWarps, 0, s>>>(p);
  } else if (vectors <= 64) {
    ln_fwd_kernel<T, RMS, 2, 1, true, SHIFTED><<<grid, 32 * kWarps, 0, s>>>(p);
  } else if (vectors <= 128) {
    ln_fwd_kernel<T, RMS, 4, 1, true, SHIFTED><<<grid, 32 * kWarps, 0, s>>>(p);
  } else if (vectors <= 4096) {
    const unsigned int threads = static_cast<unsigned int>(div_up(vectors, 128) * 32);
    ln_fwd_kernel<T, RMS, 4, 1, false, SHIFTED><<<static_cast<unsigned int>(p.N), threads, 0, s>>>(p);
  } else {
    ln_fwd_kernel<T, RMS, 8, 1, false, SHIFTED><<<static_cast<unsigned int>(p.N), 1024, 0, s>>>(p);
  }
}

template <typename T, bool RMS>
cudaError_t forward(const LnForward& p, cudaStream_t s) {
  const Fit fit = fit_of<T>(p.N, p.H, p.weight, p.bias, p.param_dtype, Matrix{p.x, p.ld_x},
                            Matrix{p.residual, p.ld_residual}, Matrix{p.y, p.ld_y}, Matrix{p.sum, p.ld_sum});
  const int64_t vectors = p.H / Vec<T>::kN;  // where rows start inside one, a few less
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
  LnForward p = {x,    residual,    weight, bias,   y, sum, mean, rstd,
                 ld_x, ld_residual, ld_y,   ld_sum, N, H,   eps,  param_dtype};
  return LN_BY_TYPE(forward, p, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
