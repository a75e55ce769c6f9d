// The optimiser's step over many tensors at once: the 2-norm of all gradients
// with the factor that clips it, and AdamW with moments in fp32 or in 8 bits.
//
// The tables of tensors travel as kernel parameters (up to 32 KB), so a call
// copies nothing to the device and can be captured in a graph.  Every element is
// read and written once: memory bandwidth bounds all of it, and with 8-bit moments,
// 16 bytes an element and some 80 instructions, the arithmetic nearly does.
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "arrival.cuh"
#include "elem.cuh"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxElems = int64_t(1) << 41;  // of one tensor
constexpr int64_t kMaxChunks = 0x7fffffff;       // of a launch

// Entries are ordered by first chunk: the one that holds chunk c.
template <typename E>
__device__ __forceinline__ int entry_of(const E* entry, int count, unsigned int c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (entry[mid].chunk0 <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------ gradient norm

constexpr int kNormChunk = 2048;  // 16-byte vectors (300 tensors of 42M bf16: 18.2 us; with 1024 20.9, with 512 23.1)
constexpr int kNormParts = 608;    // most CTAs, and partial sums, of a launch

struct NormEntry {
  const void* data;
  int64_t n;
  unsigned int chunk0;
  int dtype;
};

constexpr int kNormEntries = 1280, kNormFew = 320;
template <int MAX>
struct NormArgs {
  NormEntry entry[MAX];
  int count;
  unsigned int chunks;
  float* part;  // [gridDim.x], this launch's
  // LAST: what to make of the sums
  unsigned long long *word, tag;
  float grad_scale, max_norm, eps;
  float* out;
};

// The norm and the factor from all partial sums, added in a fixed order, by a CTA of
// kThreads.
__device__ __forceinline__ void finish_norm(const float* part, int parts, float grad_scale, float max_norm, float eps,
                                            float* out, float* scratch) {
  float sum = 0.f;
#pragma unroll 3
  for (int k = threadIdx.x; k < parts; k += kThreads) sum += __ldcg(part + k);
  sum = warp_sum(sum);
  __syncthreads();  // the scratch of an earlier sum has been read
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) sum += scratch[k];
    const float norm = sqrtf(sum) * fabsf(grad_scale);
    out[0] = norm;
    out[1] = isfinite(norm) ? grad_scale * fminf(1.f, max_norm / (norm + eps)) : __int_as_float(0x7FFFFFFF);
  }
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_finish_kernel(const float* part, int parts, float grad_scale, float max_norm, float eps, float* out) {
  __shared__ float scratch[kThreads / 32];
  grid_dependency_wait();
  finish_norm(part, parts, grad_scale, max_norm, eps, out, scratch);
}

// Most CTAs whose sums the last of them adds up itself, which saves the host a launch: a
// call with 20 tensors of 1000 takes 10.5 us so and 13.2 with a second kernel (though the
// GPU alone 4.0 and 3.0); with 608 CTAs their arrivals take longer than a second kernel
// that waits for the first (300 packed tensors 19.0 and 18.1 us).
constexpr int kMostAddedHere = 64;

// Squares of the elements in 16 bytes.
__device__ __forceinline__ float squares(const uint4& r, int dtype) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  float s = 0.f;
  if (dtype == FLCE_DTYPE_FP32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) s = fmaf(__uint_as_float(w[k]), __uint_as_float(w[k]), s);
  } else if (dtype == FLCE_DTYPE_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) s = fmaf(bf16_lo(w[k]), bf16_lo(w[k]), fmaf(bf16_hi(w[k]), bf16_hi(w[k]), s));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(reinterpret_cast<const __half2&>(w[k]));
      s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
  }
  return s;
}

// Partial sums of squares.  Memory bounds it (262M fp32: 148 us, 7.1 TB/s): four CTAs on
// an SM, each thread with eight loads under way, and one partial sum a CTA.  Each CTA
// takes a range of chunks, going from one tensor to the next.  A chunk is 16-byte
// vectors from the tensor's first 16-byte boundary on; the elements before it, and
// those after the last vector, go with the first chunk.
// LAST: the last CTA to finish adds up the sums.
template <int MAX, bool LAST>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ NormArgs<MAX> a) {
  grid_dependents_launch();
  if (LAST && blockIdx.x == 0 && threadIdx.x == 0) expect_arrivals(a.word, a.tag);
  __shared__ float scratch[kThreads / 32];
  float sum = 0.f;
  const uint64_t all = a.chunks;
  unsigned int c = static_cast<unsigned int>(all * blockIdx.x / gridDim.x);
  const unsigned int c_end = static_cast<unsigned int>(all * (blockIdx.x + 1) / gridDim.x);
  int at = entry_of(a.entry, a.count, c);
  while (c < c_end) {
    const NormEntry& e = a.entry[at];
    const unsigned int e_end = at + 1 < a.count ? a.entry[at + 1].chunk0 : a.chunks;
    const unsigned int stop = min(c_end, e_end);
    const int per = e.dtype == FLCE_DTYPE_FP32 ? 4 : 8;  // elements of a vector
    const int64_t esz = 16 / per;
    const int64_t head = min(static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(e.data) % 16) % 16) / esz, e.n);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(e.data) + head * esz);
    const int64_t vectors = (e.n - head) / per;
    const int64_t v0 = static_cast<int64_t>(c - e.chunk0) * kNormChunk;
    const int64_t v1 = min(static_cast<int64_t>(stop - e.chunk0) * kNormChunk, vectors);
    constexpr int kBatch = 8;
    int64_t i = v0 + threadIdx.x;
    for (; i < v1; i += kBatch * kThreads) {  // what is past the end counts as 0
      uint4 r[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        r[k] = i + k * kThreads < v1 ? __ldcs(v + i + k * kThreads) : make_uint4(0, 0, 0, 0);
      float batch = 0.f;  // summed apart, so that `sum` takes few additions even in a long tensor
#pragma unroll
      for (int k = 0; k < kBatch; ++k) batch += squares(r[k], e.dtype);
      sum += batch;
    }
    if (v0 == 0) {
      const int64_t tail = head + vectors * per + threadIdx.x;
      const float g = threadIdx.x < head ? load_elem(e.data, e.dtype, threadIdx.x) : 0.f;
      const float h = tail < e.n ? load_elem(e.data, e.dtype, tail) : 0.f;
      sum = fmaf(g, g, fmaf(h, h, sum));
    }
    c = stop;
    ++at;
  }
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int k = 0; k < kThreads / 32; ++k) t += scratch[k];
    a.part[blockIdx.x] = t;
  }
  if constexpr (LAST) {
    __shared__ bool last;
    if (threadIdx.x == 0) last = arrives_last(a.word, a.tag, gridDim.x);
    __syncthreads();
    if (last) finish_norm(a.part, gridDim.x, a.grad_scale, a.max_norm, a.eps, a.out, scratch);
  }
}

// -------------------------------------------------------------------- AdamW

constexpr int kAdamChunk = 4096;   // elements of a CTA
// With 8-bit moments: two blocks a warp, the second loading while the first is worked
// on, and four warps.  525M elements with a 16-bit copy took 1.42 ms so; with eight
// warps 1.52 ms, with two 1.67; with four blocks a warp 1.63, with one 1.61 (8 warps).
constexpr int kAdamChunk8 = 2048, kThreads8 = 128;
static_assert(kMaxElems / kAdamChunk8 <= kMaxChunks && kMaxElems / kAdamChunk <= kMaxChunks, "a tensor fits a launch");
static_assert(kAdamChunk8 % (FLCE_ADAMW_BLOCK * (kThreads8 / 32)) == 0, "whole blocks for every warp");
constexpr float kE4m3Max = 448.f;
constexpr unsigned int kE4m3Nan = 0x7Fu;

struct AdamEntry {
  void* param;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  void* copy;
  int64_t n;
  float lr_scale, decay;
  unsigned int chunk0;
  int index;  // place in the call's table
  int8_t param_dtype, grad_dtype, copy_dtype;
  int head;  // elements before the first vector of four in every array, or -1: the arrays differ in this
};

struct AdamNumbers {
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale_dev;
  int64_t step;
  float lr, b1, c1, b2, c2, eps;     // c = 1 - b
  float rate, correction;            // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t) when the step is known here
  float log_b1, log_b2;              // for them otherwise
  float grad_scale;
  float one, minus_zero;
  int skip_nonfinite, stochastic;
  unsigned int seed_lo, seed_hi;
};

template <int MAX>
struct AdamArgs {
  AdamEntry entry[MAX];
  int count;
  AdamNumbers num;
};

// 32 bits to 32 bits: two multiplications between shifted exclusive ors.  Every
// output bit flips with probability 0.5 +- 0.005 when any input bit does.
__device__ __forceinline__ unsigned int mix(unsigned int x) {
  x = (x ^ (x >> 16)) * 0xA54D2F6Bu;
  x = (x ^ (x >> 15)) * 0xD1B54A33u;
  return x ^ (x >> 16);
}

// Two elements' new moments.  Each product and sum rounds by itself, as the
// formulas read, so that what is then rounded to 8 bits does not depend on how
// the compiler fuses them.  It fuses products and sums of pairs whatever their
// rounding says; a fused operation whose neutral operand (-0 to add, 1 to multiply
// by) it cannot know stays by itself, at the same cost.
__device__ __forceinline__ void moments(const AdamNumbers& k, Pair g, Pair& m, Pair& v) {
  const Pair zero = pair(k.minus_zero), one = pair(k.one);
  m = fma_pair(fma_pair(m, pair(k.b1), zero), one, fma_pair(g, pair(k.c1), zero));
  v = fma_pair(fma_pair(v, pair(k.b2), zero), one, fma_pair(fma_pair(g, g, zero), pair(k.c2), zero));
}

__device__ __forceinline__ Pair sqrt_pair(Pair a) {
  const float2 f = unpair(a);
  return pair(__fsqrt_rn(f.x), __fsqrt_rn(f.y));
}

struct AdamStep {
  float factor, keep, rate, correction;
  unsigned int key;  // of this tensor and step, for the random bits
};

// The new parameters.  The divisors are 0 (with eps 0) or normal numbers (eps is at
// least the smallest, and the root of the smallest positive fp32 is 3.7e-23), as the
// approximate reciprocal needs; its error, a unit or two of 2^-23, is the update's alone.
__device__ __forceinline__ Pair updated(const AdamNumbers& k, const AdamStep& st, Pair p, Pair m, Pair root) {
  const float2 d = unpair(fma_pair(root, pair(st.correction), pair(k.eps)));
  return fma_pair(m * pair(rcp_approx(d.x), rcp_approx(d.y)), pair(-st.rate), p * pair(st.keep));
}

// Four moments over their block's scale as e4m3 numbers, the first in the lowest
// byte.  2^-120 times an e4m3 number is an fp32 number of the same exponent field,
// the normal numbers' and the subnormal ones', whose mantissa has only its upper
// three bits: bits 20 to 26 of the scaled fp32 number are the code, and the 20
// below are what rounding cuts off.  To nearest adds half of it (less one unit,
// where the code's last bit is 0, for ties to even); stochastically adds 16 random
// bits at 4 to 19, so that it rounds up with the probability of what is cut.  The
// largest, 448 but for rounding, stays below the next number either way.  (Four
// bits further left, as below, the code is the upper byte.)
//
// `random`: 32 bits an element, of which the upper half (HIGH) or the lower serves.
// KEEP (roots, not negative): what is not 0 is held as at least the smallest number.
template <bool STOCHASTIC, bool HIGH, bool KEEP>
__device__ __forceinline__ unsigned int to_e4m3_four(const Pair* x, float inverse, const unsigned int* random) {
  unsigned int t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 y2 = unpair(x[j / 2] * pair(inverse) * pair(0x1p-120f)), x2 = unpair(x[j / 2]);
    const unsigned int u = __float_as_uint(j % 2 ? y2.y : y2.x), bits = __float_as_uint(j % 2 ? x2.y : x2.x);
    unsigned int r;  // what is added, four bits to the left
    if (STOCHASTIC)
      r = __byte_perm(random[j], 0, HIGH ? 0x4324 : 0x4104);
    else
      r = (0x7FFFFu + (u >> 20 & 1u)) << 4;
    const unsigned int c = (u << 4) + r;
    if (KEEP)
      t[j] = max(c, min(bits, 0x01000000u));  // a root is 0 or far above the subnormal numbers
    else
      t[j] = (c & 0x7FFFFFFFu) | (u & 0x80000000u);
  }
  return __byte_perm(__byte_perm(t[0], t[1], 0x0073), __byte_perm(t[2], t[3], 0x0073), 0x5410);
}

__device__ __forceinline__ float from_e4m3(unsigned int code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// Four codes, lowest byte first, times the block's scale.
__device__ __forceinline__ void from_e4m3_four(unsigned int codes, float scale, Pair* out) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw raw = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(raw));
    out[h] = pair(f.x, f.y) * pair(scale);
  }
}

// A block's scale from its largest finite magnitude, and what divides by it.
__device__ __forceinline__ float block_scale(float largest, float* inverse) {
  float s = __fmul_rn(largest, 1.f / kE4m3Max);
  if (largest > 0.f) s = fmaxf(s, 0x1p-126f);
  *inverse = s > 0.f ? __frcp_rn(s) : 0.f;
  return s;
}

// Bits of |x|: they order like the numbers, infinities and NaN above all.
__device__ __forceinline__ unsigned int magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr unsigned int kInfinityBits = 0x7F800000u;

// The scale of the warp's moments x (2 N of them a lane), and what multiplies by its
// inverse.  False: some are not finite, which the scale passes over.
template <int N, bool SIGNED>
__device__ __forceinline__ bool warp_scale(const Pair* x, float* scale, float* inverse) {
  unsigned int largest = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 f = unpair(x[j]);
    const unsigned int a = SIGNED ? magnitude(f.x) : __float_as_uint(f.x);
    const unsigned int b = SIGNED ? magnitude(f.y) : __float_as_uint(f.y);
    largest = max(largest, max(a, b));
  }
  largest = __reduce_max_sync(0xffffffffu, largest);
  const bool finite = largest < kInfinityBits;
  if (!finite) {
    largest = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 f = unpair(x[j]);
      if (magnitude(f.x) < kInfinityBits) largest = max(largest, magnitude(f.x));
      if (magnitude(f.y) < kInfinityBits) largest = max(largest, magnitude(f.y));
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
  }
  *scale = block_scale(__uint_as_float(largest), inverse);
  return finite;
}

// `codes` with NaN where the four x are not finite.
__device__ __forceinline__ unsigned int mark_nan(unsigned int codes, const Pair* x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpair(x[j / 2]);
    if (magnitude(j % 2 ? f.y : f.x) >= kInfinityBits) codes = (codes & ~(0xFFu << (8 * j))) | kE4m3Nan << (8 * j);
  }
  return codes;
}

// A block of 256 elements with moments in 8 bits belongs to one warp: each lane
// holds two fours (elements 4 lane.. and 128 + 4 lane..).
constexpr int kFours = FLCE_ADAMW_BLOCK / 128, kPairs = 2 * kFours;

// Types of a tensor's parameter and gradient that are known when compiling, or not
// (kAnyType: the entry says).
constexpr int kAnyType = -1;
template <int PARAM, int GRAD>
struct Types {
  static __device__ __forceinline__ int param(const AdamEntry& e) { return PARAM == kAnyType ? e.param_dtype : PARAM; }
  static __device__ __forceinline__ int grad(const AdamEntry& e) { return GRAD == kAnyType ? e.grad_dtype : GRAD; }
};

// What a lane loads of a block.
struct Block8 {
  uint4 p[kFours], g[kFours];
  unsigned int m[kFours], r[kFours];
  float m_scale, r_scale;
};

template <typename TYPES>
__device__ __forceinline__ void load_block(const AdamEntry& e, int64_t b0, int lane, Block8& x) {
  x.m_scale = e.m_scale[b0 / FLCE_ADAMW_BLOCK];
  x.r_scale = e.v_scale[b0 / FLCE_ADAMW_BLOCK];
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const int64_t i = b0 + q * 128 + lane * 4;
    x.m[q] = __ldcs(reinterpret_cast<const unsigned int*>(static_cast<const uint8_t*>(e.m) + i));
    x.r[q] = __ldcs(reinterpret_cast<const unsigned int*>(static_cast<const uint8_t*>(e.v) + i));
    x.g[q] = load_four_bits(e.grad, TYPES::grad(e), i);
    x.p[q] = load_four_bits(e.param, TYPES::param(e), i);
  }
}

// Its step.  VECTOR: from what load_block loaded; otherwise (arrays that are not
// aligned for that, and a tensor's last block) element by element.
template <bool STOCHASTIC, bool VECTOR, typename TYPES>
__device__ __forceinline__ void step_block(const AdamEntry& e, const AdamNumbers& k, const AdamStep& st, int64_t b0,
                                           int lane, const Block8& x) {
  uint8_t* mp = static_cast<uint8_t*>(e.m);
  uint8_t* vp = static_cast<uint8_t*>(e.v);
  const int64_t block = b0 / FLCE_ADAMW_BLOCK;
  Pair m[kPairs], r[kPairs], p[kPairs], g[kPairs];
  if (VECTOR) {
#pragma unroll
    for (int q = 0; q < kFours; ++q) {
      four_pairs(x.g[q], TYPES::grad(e), g + 2 * q);
      four_pairs(x.p[q], TYPES::param(e), p + 2 * q);
      from_e4m3_four(x.m[q], x.m_scale, m + 2 * q);
      from_e4m3_four(x.r[q], x.r_scale, r + 2 * q);
    }
  } else {
    const float ms = e.m_scale[block], rs = e.v_scale[block];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      float f[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t i = b0 + (j >> 1) * 128 + lane * 4 + (j & 1) * 2 + h;
        const bool there = i < e.n;
        f[h][0] = there ? load_elem(e.param, e.param_dtype, i) : 0.f;
        f[h][1] = there ? load_elem(e.grad, e.grad_dtype, i) : 0.f;
        f[h][2] = there ? from_e4m3(mp[i]) * ms : 0.f;
        f[h][3] = there ? from_e4m3(vp[i]) * rs : 0.f;
      }
      p[j] = pair(f[0][0], f[1][0]), g[j] = pair(f[0][1], f[1][1]);
      m[j] = pair(f[0][2], f[1][2]), r[j] = pair(f[0][3], f[1][3]);
    }
  }
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    Pair v = r[j] * r[j];
    moments(k, g[j] * pair(st.factor), m[j], v);
    r[j] = sqrt_pair(v);
    p[j] = updated(k, st, p[j], m[j], r[j]);
  }
  if (VECTOR) {
#pragma unroll
    for (int q = 0; q < kFours; ++q) {
      const int64_t i = b0 + q * 128 + lane * 4;
      const float2 lo = unpair(p[2 * q]), hi = unpair(p[2 * q + 1]);
      const float4 pv = make_float4(lo.x, lo.y, hi.x, hi.y);
      store_four(e.param, TYPES::param(e), i, pv);
      if (e.copy != nullptr) store_four(e.copy, e.copy_dtype, i, pv);
    }
  }
  float m_scale, r_scale, m_inverse, r_inverse;
  const bool m_finite = warp_scale<kPairs, true>(m, &m_scale, &m_inverse);
  const bool r_finite = warp_scale<kPairs, false>(r, &r_scale, &r_inverse);
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const int64_t i = b0 + q * 128 + lane * 4;
    unsigned int random[4];
    if (STOCHASTIC) {
#pragma unroll
      for (int j = 0; j < 4; ++j) random[j] = mix((static_cast<unsigned int>(i) | j) ^ st.key);
    }
    unsigned int mc = to_e4m3_four<STOCHASTIC, true, false>(m + 2 * q, m_inverse, random);
    unsigned int rc = to_e4m3_four<STOCHASTIC, false, true>(r + 2 * q, r_inverse, random);
    if (!m_finite) mc = mark_nan(mc, m + 2 * q);
    if (!r_finite) rc = mark_nan(rc, r + 2 * q);
    if (VECTOR) {
      __stcs(reinterpret_cast<unsigned int*>(mp + i), mc);
      __stcs(reinterpret_cast<unsigned int*>(vp + i), rc);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < e.n) {
          const float2 two = unpair(p[2 * q + j / 2]);
          store_elem(e.param, e.param_dtype, i + j, j % 2 ? two.y : two.x);
          if (e.copy != nullptr) store_elem(e.copy, e.copy_dtype, i + j, j % 2 ? two.y : two.x);
          mp[i + j] = static_cast<uint8_t>(mc >> (8 * j));
          vp[i + j] = static_cast<uint8_t>(rc >> (8 * j));
        }
    }
  }
  __syncwarp();  // every lane has read the old scales
  if (lane == 0) {
    e.m_scale[block] = m_scale;
    e.v_scale[block] = r_scale;
  }
}

// The numbers of one tensor's step; false: it is to be skipped.
__device__ __forceinline__ bool step_numbers(const AdamEntry& e, const AdamNumbers& k, AdamStep& st) {
  st.factor = k.grad_scale_dev != nullptr ? *k.grad_scale_dev : k.grad_scale;
  const float lr = (k.lr_dev != nullptr ? *k.lr_dev : k.lr) * e.lr_scale;
  float rate = k.rate;
  st.correction = k.correction;
  int64_t step = k.step;
  if (k.step_dev != nullptr) {  // 1 - b^t = -(e^(t ln b) - 1), without the cancellation
    step = *k.step_dev;
    rate = 1.f / -expm1f(static_cast<float>(step) * k.log_b1);
    st.correction = rsqrtf(-expm1f(static_cast<float>(step) * k.log_b2));
  }
  st.rate = rate * lr;
  st.keep = 1.f - lr * e.decay;
  st.key = mix(k.seed_lo);
  st.key = mix(st.key ^ k.seed_hi);
  st.key = mix(st.key ^ static_cast<unsigned int>(step));
  st.key = mix(st.key ^ static_cast<unsigned int>(e.index));
  return !k.skip_nonfinite || isfinite(st.factor);
}

// Tensors with fp32 moments: 28 bytes an element (fp32 parameter and gradient, 30 with
// a 16-bit copy) and about 40 instructions, so memory bounds it: 262M elements with a
// copy take 1.13 ms, 7.0 TB/s, as fast as a plain copy.  A thread takes four elements
// of every array at a time, four times; 32 registers let every SM hold 64 warps, whose
// loads cover the latency without looking ahead.  What is left at a tensor's ends goes
// one by one, and so does all of a tensor whose arrays lie at different boundaries: 134M
// elements with bf16 gradients 758 us instead of 543 (8-bit moments 827 instead of 312).
template <int MAX>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamArgs<MAX> a) {
  const AdamEntry& e = a.entry[entry_of(a.entry, a.count, blockIdx.x)];
  const AdamNumbers& k = a.num;
  AdamStep st;
  if (!step_numbers(e, k, st)) return;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x - e.chunk0) * kAdamChunk;
  float* mp = static_cast<float*>(e.m);
  float* vp = static_cast<float*>(e.v);
  const auto one = [&](int64_t i) {
    Pair m = pair(mp[i]), v = pair(vp[i]);
    moments(k, pair(load_elem(e.grad, e.grad_dtype, i) * st.factor), m, v);
    const float p = unpair(updated(k, st, pair(load_elem(e.param, e.param_dtype, i)), m, sqrt_pair(v))).x;
    mp[i] = unpair(m).x;
    vp[i] = unpair(v).x;
    store_elem(e.param, e.param_dtype, i, p);
    if (e.copy != nullptr) store_elem(e.copy, e.copy_dtype, i, p);
  };
  if (e.head < 0) {
    const int64_t i1 = min(i0 + kAdamChunk, e.n);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) one(i);
    return;
  }
  // vectors of four from element `head` on
  const int64_t whole = e.n - (e.n - e.head) % 4;
  for (int64_t i = i0 + e.head + threadIdx.x * 4; i < min(i0 + e.head + kAdamChunk, whole); i += kThreads * 4) {
    float4 m = __ldcs(reinterpret_cast<const float4*>(mp + i)), v = __ldcs(reinterpret_cast<const float4*>(vp + i));
    const uint4 pb = load_four_bits(e.param, e.param_dtype, i), gb = load_four_bits(e.grad, e.grad_dtype, i);
    float4 p = four_floats(pb, e.param_dtype);
    const float4 g = four_floats(gb, e.grad_dtype);
    const auto part = [&](float& p0, float& p1, float g0, float g1, float& m0, float& m1, float& v0, float& v1) {
      Pair m2 = pair(m0, m1), v2 = pair(v0, v1);
      moments(k, pair(g0, g1) * pair(st.factor), m2, v2);
      const float2 pf = unpair(updated(k, st, pair(p0, p1), m2, sqrt_pair(v2))), mf = unpair(m2), vf = unpair(v2);
      p0 = pf.x, p1 = pf.y, m0 = mf.x, m1 = mf.y, v0 = vf.x, v1 = vf.y;
    };
    part(p.x, p.y, g.x, g.y, m.x, m.y, v.x, v.y);
    part(p.z, p.w, g.z, g.w, m.z, m.w, v.z, v.w);
    __stcs(reinterpret_cast<float4*>(mp + i), m);
    __stcs(reinterpret_cast<float4*>(vp + i), v);
    store_four(e.param, e.param_dtype, i, p);
    if (e.copy != nullptr) store_four(e.copy, e.copy_dtype, i, p);
  }
  if (i0 == 0 && threadIdx.x < e.head) one(threadIdx.x);
  if (whole + threadIdx.x < e.n && whole < i0 + e.head + kAdamChunk && whole >= i0 + e.head) one(whole + threadIdx.x);
}

// A warp takes blocks, and has the next one's loads under way while it works on one:
// the two maxima over the block and the roundings behind them are a long chain.
template <bool STOCHASTIC, typename TYPES>
__device__ __forceinline__ void step_chunk(const AdamEntry& e, const AdamNumbers& k) {
  constexpr int64_t kStep = kThreads8 / 32 * FLCE_ADAMW_BLOCK;
  const int lane = threadIdx.x & 31;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x - e.chunk0) * kAdamChunk8, i1 = min(i0 + kAdamChunk8, e.n);
  // where blocks by vectors end
  const int64_t whole = e.head == 0 ? min(i1, e.n - e.n % FLCE_ADAMW_BLOCK) : 0;
  int64_t b0 = i0 + (threadIdx.x >> 5) * FLCE_ADAMW_BLOCK;
  Block8 next;
  if (b0 < whole) load_block<TYPES>(e, b0, lane, next);
  AdamStep st;
  if (!step_numbers(e, k, st)) return;
  st.key = mix(st.key ^ static_cast<unsigned int>(static_cast<uint64_t>(i0) >> 32));  // the whole chunk's
  for (; b0 < whole; b0 += kStep) {
    const Block8 now = next;
    if (b0 + kStep < whole) load_block<TYPES>(e, b0 + kStep, lane, next);
    step_block<STOCHASTIC, true, TYPES>(e, k, st, b0, lane, now);
  }
  for (; b0 < i1; b0 += kStep) step_block<STOCHASTIC, false, Types<kAnyType, kAnyType>>(e, k, st, b0, lane, next);
}

// Tensors with 8-bit moments.  What the arithmetic issues bounds this as closely as
// memory does, so fp32 parameters, the master weights that such moments go with, have
// code of their own for the gradients that FLCE (fp32) and a 16-bit model (bf16) leave:
// 268M elements with a 16-bit copy, to nearest, take 716 and 621 us so and 774 and 739 by
// the code for any types.  By that, fp16 gradients take 747 us and bf16 parameters and
// gradients 663 (741 and 660 if the kernel has no other code).  Eight CTAs on an SM: 525M
// elements with a 16-bit copy took 1.36 ms so (7.0 TB/s), 1.43 with seven, 1.48 with
// six, 1.59 with five (the 90 registers it would take by itself).
template <int MAX, bool STOCHASTIC>
__global__ void __launch_bounds__(kThreads8, 8) adamw8_kernel(const __grid_constant__ AdamArgs<MAX> a) {
  const AdamEntry& e = a.entry[entry_of(a.entry, a.count, blockIdx.x)];
  if (e.param_dtype == FLCE_DTYPE_FP32 && e.grad_dtype == FLCE_DTYPE_FP32)
    step_chunk<STOCHASTIC, Types<FLCE_DTYPE_FP32, FLCE_DTYPE_FP32>>(e, a.num);
  else if (e.param_dtype == FLCE_DTYPE_FP32 && e.grad_dtype == FLCE_DTYPE_BF16)
    step_chunk<STOCHASTIC, Types<FLCE_DTYPE_FP32, FLCE_DTYPE_BF16>>(e, a.num);
  else
    step_chunk<STOCHASTIC, Types<kAnyType, kAnyType>>(e, a.num);
}

template <int MAX>
cudaError_t launch_norm(const NormEntry* entry, const NormArgs<1>& rest, int grid, cudaStream_t s) {
  NormArgs<MAX> a;
  std::copy(entry, entry + rest.count, a.entry);
  a.count = rest.count;
  a.chunks = rest.chunks;
  a.part = rest.part;
  a.word = rest.word;
  a.tag = rest.tag;
  a.grad_scale = rest.grad_scale;
  a.max_norm = rest.max_norm;
  a.eps = rest.eps;
  a.out = rest.out;
  prof_begin(s, FLCE_KERNEL_GRAD_NORM);
  if (a.word != nullptr)
    grad_norm_kernel<MAX, true><<<grid, kThreads, 0, s>>>(a);
  else
    grad_norm_kernel<MAX, false><<<grid, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  prof_end(s);
  return e;
}

template <int MAX>
cudaError_t launch_adamw(const AdamEntry* entry, int count, unsigned int chunks, const AdamNumbers& num, int bits,
                         cudaStream_t s) {
  AdamArgs<MAX> a;
  std::copy(entry, entry + count, a.entry);
  a.count = count;
  a.num = num;
  prof_begin(s, FLCE_KERNEL_ADAMW);
  if (bits == 32)
    adamw_kernel<MAX><<<chunks, kThreads, 0, s>>>(a);
  else if (num.stochastic)
    adamw8_kernel<MAX, true><<<chunks, kThreads8, 0, s>>>(a);
  else
    adamw8_kernel<MAX, false><<<chunks, kThreads8, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  prof_end(s);
  return e;
}

// Tables of a few sizes, the largest what kernel parameters hold and each other a third
// or a quarter of the next: a launch copies its whole parameter block, 32 KB of it in a
// microsecond.  Steps of small tensors, the C call alone: 100 of them 4.4 us from the
// table of 128 and 5.4 from that of 360, 16 of them 4.2 from the table of 40 and 4.5; the
// norm of 100 gradients 5.9 us from the table of 320 and 7.0 from that of 1280.  Smaller
// tables still gained nothing (4 entries 4.14 against 4.15, 16 of the norm's 6.22 and 6.26).
constexpr int kAdamEntries = 360, kAdamMore = 128, kAdamFew = 40;
static_assert(sizeof(AdamArgs<kAdamEntries>) <= 32764, "kernel parameters");
static_assert(sizeof(NormArgs<kNormEntries>) <= 32764, "kernel parameters");

cudaError_t launch_norm_any(const NormEntry* entry, const NormArgs<1>& rest, int grid, cudaStream_t s) {
  if (rest.count <= kNormFew) return launch_norm<kNormFew>(entry, rest, grid, s);
  return launch_norm<kNormEntries>(entry, rest, grid, s);
}

cudaError_t launch_adamw_any(const AdamEntry* entry, int count, unsigned int chunks, const AdamNumbers& num, int bits,
                             cudaStream_t s) {
  if (count <= kAdamFew) return launch_adamw<kAdamFew>(entry, count, chunks, num, bits, s);
  if (count <= kAdamMore) return launch_adamw<kAdamMore>(entry, count, chunks, num, bits, s);
  return launch_adamw<kAdamEntries>(entry, count, chunks, num, bits, s);
}

// Elements before every array's first boundary of four, where that is the same
// for all of them; else -1.  (Blocks of 8-bit moments are counted from the
// start, so that only 0 serves there.)
int common_head(const flce_adamw_tensor_t& t) {
  const int state = t.moment_bits == 8 ? 0 : 2;  // log2 of an element's size
  const auto size = [](int dtype) { return dtype == FLCE_DTYPE_FP32 ? 2 : 1; };
  const auto before = [](const void* p, int log2_size) {
    return static_cast<int>(-(reinterpret_cast<uintptr_t>(p) >> log2_size) & 3);
  };
  const int head = before(t.param, size(t.param_dtype));
  if (head != before(t.grad, size(t.grad_dtype)) || head != before(t.exp_avg, state) ||
      head != before(t.exp_avg_sq, state) || (t.copy != nullptr && head != before(t.copy, size(t.copy_dtype))))
    return -1;
  return t.n > head ? head : -1;
}

// At least the vectors from the first boundary on (a chunk too many finds nothing).
int64_t norm_chunks(const flce_tensor_t& t) {
  return div_up(t.n, kNormChunk * static_cast<int64_t>(16 / elem_size(t.dtype)));
}

// The partial sums of every launch, then the word that finds the last CTA.
size_t norm_parts_bytes(int64_t count) {
  return align_up(static_cast<size_t>(std::max<int64_t>(1, div_up(count, kNormEntries))) * kNormParts * 4, 256);
}
size_t norm_workspace(int64_t count) { return norm_parts_bytes(count) + 256; }

flce_status_t check_tensor(const flce_adamw_tensor_t& t) {
  if (t.n < 0 || t.n > kMaxElems) return FLCE_ERR_INVALID_ARG;
  if (!float_dtype(t.param_dtype) || !float_dtype(t.grad_dtype) || (t.copy != nullptr && !float_dtype(t.copy_dtype)))
    return FLCE_ERR_UNSUPPORTED;
  if (t.moment_bits != 8 && t.moment_bits != 32) return FLCE_ERR_UNSUPPORTED;
  if (!isfinite(t.lr_scale) || !isfinite(t.weight_decay)) return FLCE_ERR_INVALID_ARG;
  if (t.n == 0) return FLCE_OK;
  if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr)
    return FLCE_ERR_INVALID_ARG;
  const bool scaled = t.moment_bits == 8;
  if (scaled != (t.exp_avg_scale != nullptr) || scaled != (t.exp_avg_sq_scale != nullptr)) return FLCE_ERR_INVALID_ARG;
  const size_t state = scaled ? 1 : 4;
  if (!aligned_to(t.param, elem_size(t.param_dtype)) || !aligned_to(t.grad, elem_size(t.grad_dtype)) ||
      (t.copy != nullptr && !aligned_to(t.copy, elem_size(t.copy_dtype))) || !aligned_to(t.exp_avg, state) ||
      !aligned_to(t.exp_avg_sq, state) || !aligned_to(t.exp_avg_scale, 4) || !aligned_to(t.exp_avg_sq_scale, 4))
    return FLCE_ERR_MISALIGNED;
  return FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

size_t grad_norm_workspace_size(int64_t count) { return count < 0 ? 0 : norm_workspace(count); }

flce_status_t grad_norm(const flce_tensor_t* tensors, int64_t count, float grad_scale, float max_norm, float eps,
                        float* out, void* workspace, size_t workspace_bytes, flce_stream_t stream_) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (count < 0 || (count > 0 && tensors == nullptr) || out == nullptr) return FLCE_ERR_INVALID_ARG;
  if (!isfinite(grad_scale) || !(max_norm >= 0.f) || !(eps >= 0.f) || isinf(eps)) return FLCE_ERR_INVALID_ARG;
  int64_t all = 0;
  for (int64_t i = 0; i < count; ++i) {
    const flce_tensor_t& t = tensors[i];
    if (t.n < 0 || t.n > kMaxElems || (t.n > 0 && t.data == nullptr)) return FLCE_ERR_INVALID_ARG;
    if (!float_dtype(t.dtype)) return FLCE_ERR_UNSUPPORTED;
    if (!aligned_to(t.data, elem_size(t.dtype))) return FLCE_ERR_MISALIGNED;
    // together they fit one launch's numbers, so that only their count makes launches, as the workspace has it
    all += norm_chunks(t);
    if (all > kMaxChunks) return FLCE_ERR_INVALID_ARG;
  }
  if (!aligned_to(out, 4)) return FLCE_ERR_MISALIGNED;
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < norm_workspace(count))
    return FLCE_ERR_WORKSPACE;
  const int most = std::min(kNormParts, 4 * device_sm_count());
  NormEntry entry[kNormEntries];
  NormArgs<1> rest = {};
  float* const part = static_cast<float*>(workspace);
  int parts = 0;
  rest.tag = next_arrival_tag();
  rest.grad_scale = grad_scale;
  rest.max_norm = max_norm;
  rest.eps = eps;
  rest.out = out;
  int64_t i = 0;
  const auto skip_empty = [&] {
    while (i < count && tensors[i].n == 0) ++i;
  };
  skip_empty();
  do {  // once at least: no tensors have a norm too
    int64_t chunks = 0;
    rest.count = 0;
    while (i < count && rest.count < kNormEntries) {
      entry[rest.count++] = {tensors[i].data, tensors[i].n, static_cast<unsigned int>(chunks), tensors[i].dtype};
      chunks += norm_chunks(tensors[i]);
      ++i;
      skip_empty();
    }
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, most)));
    rest.chunks = static_cast<unsigned int>(chunks);
    rest.part = part + parts;
    if (parts == 0 && i >= count && grid <= kMostAddedHere)
      rest.word = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) + norm_parts_bytes(count));
    if (launch_norm_any(entry, rest, grid, s) != cudaSuccess) return FLCE_ERR_CUDA;
    parts += grid;
  } while (i < count);
  if (rest.word != nullptr) return FLCE_OK;
  prof_begin(s, FLCE_KERNEL_GRAD_NORM);
  const cudaError_t e = launch_after(grad_norm_finish_kernel, dim3(1), dim3(kThreads), s,
                                     static_cast<const float*>(part), parts, grad_scale, max_norm, eps, out);
  prof_end(s);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

flce_status_t adamw_step(const flce_adamw_tensor_t* tensors, int64_t count, const flce_adamw_t* numbers,
                         flce_stream_t stream_) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (numbers == nullptr || count < 0 || count > 0x7fffffff || (count > 0 && tensors == nullptr))
    return FLCE_ERR_INVALID_ARG;
  const flce_adamw_t& u = *numbers;
  if (!(u.beta1 >= 0 && u.beta1 < 1 && u.beta2 >= 0 && u.beta2 < 1) || !(u.eps >= 0) || !isfinite(u.eps))
    return FLCE_ERR_INVALID_ARG;
  if ((u.lr_dev == nullptr && !isfinite(u.lr)) || (u.step_dev == nullptr && u.step < 1)) return FLCE_ERR_INVALID_ARG;
  if ((u.skip_nonfinite != 0 && u.skip_nonfinite != 1) || (u.stochastic != 0 && u.stochastic != 1))
    return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(u.step_dev, 8) || !aligned_to(u.lr_dev, 4) || !aligned_to(u.grad_scale_dev, 4))
    return FLCE_ERR_MISALIGNED;
  for (int64_t i = 0; i < count; ++i) {
    const flce_status_t st = check_tensor(tensors[i]);
    if (st != FLCE_OK) return st;
  }
  const double t = static_cast<double>(u.step);
  AdamNumbers num = {};
  num.step_dev = u.step_dev;
  num.lr_dev = u.lr_dev;
  num.grad_scale_dev = u.grad_scale_dev;
  num.step = u.step;
  num.lr = static_cast<float>(u.lr);
  num.b1 = static_cast<float>(u.beta1);
  num.c1 = static_cast<float>(1 - u.beta1);
  num.b2 = static_cast<float>(u.beta2);
  num.c2 = static_cast<float>(1 - u.beta2);
  // at least the smallest normal number (the reciprocal's input), far below any root that is not 0: a parameter whose
  // moments are 0 stays where it is
  num.eps = u.eps > 0 ? std::max(static_cast<float>(u.eps), 0x1p-126f) : 0.f;
  num.log_b1 = static_cast<float>(log(u.beta1));
  num.log_b2 = static_cast<float>(log(u.beta2));
  num.rate = static_cast<float>(1 / (1 - pow(u.beta1, t)));
  num.correction = static_cast<float>(1 / sqrt(1 - pow(u.beta2, t)));
  num.grad_scale = u.grad_scale;
  num.one = 1.f;
  num.minus_zero = -0.f;
  num.skip_nonfinite = u.skip_nonfinite;
  num.stochastic = u.stochastic;
  num.seed_lo = static_cast<unsigned int>(u.seed);
  num.seed_hi = static_cast<unsigned int>(u.seed >> 32);
  AdamEntry entry[kAdamEntries];
  for (const int bits : {32, 8}) {
    for (int64_t i = 0; i < count;) {
      int filled = 0;
      int64_t chunks = 0;
      for (; i < count && filled < kAdamEntries; ++i) {
        const flce_adamw_tensor_t& x = tensors[i];
        if (x.n == 0 || x.moment_bits != bits) continue;
        const int head = common_head(x);
        const int64_t more = bits == 8 ? div_up(x.n, kAdamChunk8) : div_up(head > 0 ? x.n - head : x.n, kAdamChunk);
        if (chunks + more > kMaxChunks) break;  // the next launch's: by itself every tensor fits
        entry[filled++] = {x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale, x.copy, x.n,
                           x.lr_scale, x.weight_decay, static_cast<unsigned int>(chunks), static_cast<int>(i),
                           static_cast<int8_t>(x.param_dtype), static_cast<int8_t>(x.grad_dtype),
                           static_cast<int8_t>(x.copy_dtype), head};
        chunks += more;
      }
      if (filled == 0) break;
      if (launch_adamw_any(entry, filled, static_cast<unsigned int>(chunks), num, bits, s) != cudaSuccess)
        return FLCE_ERR_CUDA;
    }
  }
  return FLCE_OK;
}

}  // extern "C"
