// Layer norm, and its form without the mean (rms), in front of the head: the
// backward pass, with the column sums that give the weight's and the bias's
// gradient.
//
// Every element is moved once (3 N H b bytes, 4 N H b with the gradient of the
// residual stream), with about fifteen operations on it: memory bandwidth bounds it.
#include <math.h>

#include <atomic>

#include "arrival.cuh"
#include "norm.cuh"

namespace flce {
namespace {

// Column sums of the backward pass are taken by at most this many CTAs, each
// leaving one partial row of H sums (the workspace holds them all).
constexpr int kMaxParts = 304;

// Elements between partial rows: they are read by fours.
__host__ __device__ inline int64_t part_ld(int64_t H) { return (H + 3) / 4 * 4; }

struct LnBackward {
  const void *grad_y, *x, *weight, *grad_sum;
  const float *mean, *rstd;
  void* grad_x;
  int64_t ld_grad_y, ld_x, ld_grad_sum, ld_grad_x, N, H;
  int param_dtype;
  float2* row_terms;       // [N]: mean(u), mean(u xhat), of the form by elements
  float *part_w, *part_b;  // [parts][part_ld(H)]
  int parts;
  float *grad_weight, *grad_bias;
  int accumulate;
  unsigned long long *word, tag;  // of a launch whose last CTA adds up the partial rows (else null)
};

// ------------------------------------------------------- rows by 16-byte vectors

// 16 bytes from global to shared memory, without a register between; the thread
// that issued it sees them after copies_arrived.
__device__ __forceinline__ void copy_16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>
__device__ __forceinline__ void copies_arrived() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory");
}

__device__ __forceinline__ uint4 load_shared(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}

__device__ __forceinline__ void load_pairs(uint32_t a, Pair& x, Pair& y) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x.v), "=l"(y.v) : "r"(a) : "memory");
}
__device__ __forceinline__ void store_pairs(uint32_t a, Pair x, Pair y) {
  asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(a), "l"(x.v), "l"(y.v) : "memory");
}

// A barrier of `threads` threads (whole warps) of the CTA; 0 is __syncthreads'.
__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Threads of a CTA, one CTA on each SM: 112 registers each, which leaves the kernel
// that adds up the CTAs' sums 8192 (128 where a bias's sums need more).  What a row
// costs a thread beside its elements (addresses, sums, a barrier) is as much as eight
// elements do, so a thread takes two vectors rather than there being twice as many
// threads: at [16384, 4096] in bf16 with one vector each 5000 instructions a row, near
// all that the SM can issue while memory moves it.
constexpr int kBwdThreads = 512;

// Whether the weights lie in shared memory: where the sums for a bias with the tests
// for missing vectors, or the column beside the vectors, take the registers.  (Spilled
// ones cost far more, as next to the ring the first-level cache has room for little:
// bf16 [20000, 1001] took 72 us with 56 bytes a thread spilled and 42 so.)
template <typename T, int VPT>
constexpr bool share_weights(bool bias, bool shifted, bool full) {
  return sizeof(T) == 2 && VPT == 2 && (shifted || (bias && !full));
}

// Groups of more than a warp have a named barrier each (1 to 15).
constexpr int kMaxBarriers = 15;

// Sums over LANES lanes of a warp (aligned groups of 32, 16 or 8, which may have come
// here at different times), to all of them.
template <int LANES>
__device__ __forceinline__ unsigned int lanes_mask() {
  return LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  const unsigned int mask = lanes_mask<LANES>();
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}
// Both numbers' with one exchange more than for one: the lower half of the lanes goes
// on with the first, the upper half with the second.
template <int LANES>
__device__ __forceinline__ float2 lanes_sum2(float2 v) {
  const unsigned int mask = lanes_mask<LANES>();
  const bool upper = threadIdx.x & (LANES / 2);
  float mine = upper ? v.y : v.x;
  mine += __shfl_xor_sync(mask, upper ? v.x : v.y, LANES / 2);
#pragma unroll
  for (int o = LANES / 4; o > 0; o >>= 1) mine += __shfl_xor_sync(mask, mine, o);
  const float other = __shfl_xor_sync(mask, mine, LANES / 2);
  return upper ? make_float2(other, mine) : make_float2(mine, other);
}

// The launch's last CTA adds up the partial rows.
__device__ __forceinline__ void add_up_here(const LnBackward& p) {
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) last = arrives_last(p.word, p.tag, gridDim.x);
  __syncthreads();
  if (!last) return;
  // four columns of one of the two sums for a thread, most of its loads under way at once
  const int fours = static_cast<int>(part_ld(p.H) / 4);
  for (int item = threadIdx.x; item < 2 * fours; item += blockDim.x) {
    const bool weight = item < fours;
    float* const out = weight ? p.grad_weight : p.grad_bias;
    if (out == nullptr) continue;
    const int c = (weight ? item : item - fours) * 4;
    const float* const part = (weight ? p.part_w : p.part_b) + c;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
    for (unsigned int k = 0; k < gridDim.x; ++k) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part + k * part_ld(p.H)));
      a[0] += v.x, a[1] += v.y, a[2] += v.z, a[3] += v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < p.H) out[c + i] = p.accumulate ? out[c + i] + a[i] : a[i];
  }
}

// grad_x and column sums, with
//   u = grad_y weight,  grad_x = rstd (u - mean(u) - xhat mean(u xhat)) + grad_sum,
// the means over a row, and the columns' sums of grad_y xhat and grad_y over the rows.
// Memory bounds it: bf16 [16384, 4096] without a mean, with grad_sum, takes 80 us (6.7
// TB/s; 85 us with the kernel that adds up the sums, and a plain copy of as many bytes
// 86), fp32 [8191, 2048] 37 us (5.5 TB/s; a copy 37).  `group` threads take a row, VPT
// vectors each, and a CTA holds as many such groups as fit.  A thread keeps its columns
// from row to row, so that the sums over the rows stay in its registers until the end;
// so where rows start inside a vector, a group takes only rows that start at the same
// place (every eighth, or every fourth fp32 one).  Rows are fetched DEPTH - 1 ahead into
// shared memory by asynchronous copies, each thread its own vectors: nothing waits for
// another thread but the two sums over the row.  LANES: those of a warp that a row takes
// (32 where it takes whole warps).
//
// FULL: every thread has all of its vectors (the usual widths), so nothing asks.
// LAST: for few rows, the launch's last CTA adds up the CTAs' sums (kernels of their
// own: with that code in it the rows' loop took 8 % longer).
template <typename T, bool RMS, bool BIAS, int VPT, int LANES, int DEPTH, bool SHIFTED, bool FULL, bool LAST>
__global__ void __maxnreg__((VPT > 2 || (sizeof(T) == 2 && (BIAS || SHIFTED)) ? 128 : 112))
    ln_bwd_kernel(const LnBackward p, int group, int groups) {
  constexpr bool kShareWeights = share_weights<T, VPT>(BIAS, SHIFTED, FULL);
  using V = Vec<T>;
  constexpr int kN = V::kN, kP = kN / 2;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float2 scratch[2][kMaxBarriers][32];
  const int in_cta = threadIdx.x / group, t = threadIdx.x % group, lane = threadIdx.x & 31;
  const int warps = group >> 5, warp = t >> 5;
  // rows n0, n0 + step, ... (SHIFTED: step is a multiple of kN)
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * groups + in_cta;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const Row<T, SHIFTED> row(static_cast<const T*>(p.x) + n0 * p.ld_x, p.H);
  const auto has = [&](int k) { return FULL || t + k * group < row.vectors; };  // whether there is a k-th vector
  const int arrays = p.grad_sum != nullptr ? 3 : 2;
  const uint32_t vector_bytes = blockDim.x * 16, array_bytes = vector_bytes * VPT, stage_bytes = array_bytes * arrays;
  // shared memory: the weights where they lie there, then the ring
  const uint32_t my_weights = smem_addr(ring) + threadIdx.x * 16;
  const uint32_t mine = my_weights + (kShareWeights ? 2 * array_bytes : 0);
  // this thread's first vector of the next row to fetch, in each array
  const int64_t lane_offset = row.column(t);
  const T* next_g = static_cast<const T*>(p.grad_y) + n0 * p.ld_grad_y + lane_offset;
  const T* next_x = static_cast<const T*>(p.x) + n0 * p.ld_x + lane_offset;
  const T* next_s = static_cast<const T*>(p.grad_sum) + n0 * p.ld_grad_sum + lane_offset;
  const auto fetch_array = [&](int64_t ld, const T*& vector, uint32_t to) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (has(k)) copy_16(to + k * vector_bytes, vector + k * group * kN);
    vector += step * ld;
  };
  const auto fetch = [&](uint32_t stage) {
    fetch_array(p.ld_grad_y, next_g, mine + stage);
    fetch_array(p.ld_x, next_x, mine + stage + array_bytes);
    if (arrays == 3) fetch_array(p.ld_grad_sum, next_s, mine + stage + 2 * array_bytes);
  };
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) {
    if (n0 + d * step < p.N) fetch(d * stage_bytes);
    copies_issued();
  }
  grid_dependents_launch();
  if (LAST && blockIdx.x == 0 && threadIdx.x == 0) expect_arrivals(p.word, p.tag);

  Pair sw[VPT][kP], sb[VPT][kP], w[VPT][kP];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int i = 0; i < kP; ++i) sw[k][i] = sb[k][i] = pair(0.f);
  // kept with one or two vectors a thread, in registers or (kShareWeights) in this
  // thread's part of shared memory; with more read again
  constexpr bool kKeep = VPT <= 2;
  // whether u and xhat are formed again for grad_x instead of being kept over the barrier
  constexpr bool kAgain = !kKeep || (kShareWeights && BIAS && SHIFTED);
  const auto weights = [&](int k) {
    float f[kN];
    if (p.weight != nullptr && has(k)) {
      row.params(p.weight, p.param_dtype, t + k * group, f);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) w[k][i] = pair(f[2 * i], f[2 * i + 1]);
  };
  if (kKeep) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      weights(k);
      if (kShareWeights) {
#pragma unroll
        for (int i = 0; i < kP; i += 2) store_pairs(my_weights + (k * kP + i) / 2 * vector_bytes, w[k][i], w[k][i + 1]);
      }
    }
  }
  const auto elements = [&](uint32_t stage, int array, int k, Pair* f2) {
    float f[kN];
    V::unpack(load_shared(mine + stage + array * array_bytes + k * vector_bytes), f);
#pragma unroll
    for (int i = 0; i < kP; ++i) f2[i] = pair(f[2 * i], f[2 * i + 1]);
  };
  const float over = 1.f / static_cast<float>(p.H);
  // SHIFTED: the element beside the vectors, loaded a row ahead like the row's statistics
  const int c_extra = row.extra(t);
  const T* extra_g = static_cast<const T*>(p.grad_y) + n0 * p.ld_grad_y + c_extra;
  const T* extra_x = static_cast<const T*>(p.x) + n0 * p.ld_x + c_extra;
  const T* extra_s = static_cast<const T*>(p.grad_sum) + n0 * p.ld_grad_sum + c_extra;
  const float w_extra = c_extra >= 0 && p.weight != nullptr ? load_elem(p.weight, p.param_dtype, c_extra) : 1.f;
  float sw_extra = 0.f, sb_extra = 0.f;
  float next_mu = 0.f, next_inv = 0.f;
  T next_ge = from_float<T>(0.f), next_xe = next_ge, next_se = next_ge;
  const auto ahead = [&](int64_t n) {
    next_mu = RMS ? 0.f : p.mean[n];
    next_inv = p.rstd[n];
    if (c_extra >= 0) {
      next_ge = *extra_g;
      next_xe = *extra_x;
      if (arrays == 3) next_se = *extra_s;
    }
    if (SHIFTED) {
      extra_g += step * p.ld_grad_y;
      extra_x += step * p.ld_x;
      extra_s += step * p.ld_grad_sum;
    }
  };
  if (n0 < p.N) ahead(n0);
  uint32_t stage = 0;
  const uint32_t last_stage = (DEPTH - 1) * stage_bytes;
  int turn = 0;
  T* to = static_cast<T*>(p.grad_x) + n0 * p.ld_grad_x;
  for (int64_t n = n0; n < p.N; n += step) {
    const float mu = next_mu, inv = next_inv;
    const T ge = next_ge, xe = next_xe, se = next_se;
    if (n + step < p.N) ahead(n + step);
    copies_arrived<DEPTH - 2>();
    // the next row to fetch goes where this thread's part of the row before this one was
    if (n + (DEPTH - 1) * step < p.N) fetch(stage == 0 ? last_stage : stage - stage_bytes);
    copies_issued();
    Pair g[VPT][kP], xhat[VPT][kP];  // g: grad_y, then u
    const auto read = [&](int k) {
      elements(stage, 0, k, g[k]);
      elements(stage, 1, k, xhat[k]);
      if (!kKeep) weights(k);
      if (kShareWeights) {
#pragma unroll
        for (int i = 0; i < kP; i += 2) load_pairs(my_weights + (k * kP + i) / 2 * vector_bytes, w[k][i], w[k][i + 1]);
      }
#pragma unroll
      for (int i = 0; i < kP; ++i)
        xhat[k][i] = RMS ? xhat[k][i] * pair(inv) : (xhat[k][i] + pair(-mu)) * pair(inv);
    };
    Pair s1 = pair(0.f), s2 = pair(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (has(k)) {
        read(k);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          sw[k][i] = fma_pair(g[k][i], xhat[k][i], sw[k][i]);
          if (BIAS) sb[k][i] = sb[k][i] + g[k][i];
          g[k][i] = g[k][i] * w[k][i];
          if (!RMS) s1 = s1 + g[k][i];
          s2 = fma_pair(g[k][i], xhat[k][i], s2);
        }
      }
    }
    const float2 f1 = unpair(s1), f2 = unpair(s2);
    float2 s = make_float2(f1.x + f1.y, f2.x + f2.y);
    float u_extra = 0.f, xhat_extra = 0.f;
    if (c_extra >= 0) {
      xhat_extra = (to_float(xe) - mu) * inv;
      sw_extra = fmaf(to_float(ge), xhat_extra, sw_extra);
      sb_extra += to_float(ge);
      u_extra = to_float(ge) * w_extra;
      s.x += u_extra;
      s.y = fmaf(u_extra, xhat_extra, s.y);
    }
    if (RMS)
      s.y = lanes_sum<LANES>(s.y);
    else
      s = lanes_sum2<LANES>(s);
    if (LANES == 32 && warps > 1) {
      // one barrier a row: the scratch of a row is written again two rows later
      if (lane == 0) scratch[turn][in_cta][warp] = s;
      group_barrier(1 + in_cta, group);
      s = lane < warps ? scratch[turn][in_cta][lane] : make_float2(0.f, 0.f);
      if (RMS)
        s.y = lanes_sum<32>(s.y);
      else
        s = lanes_sum2<32>(s);
      turn ^= 1;
    }
    if (p.grad_x != nullptr) {
      // (u - mean(u) - xhat mean(u xhat)) rstd + grad_sum
      const Pair c1 = pair(-s.x * over * inv), c2 = pair(-s.y * over * inv);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int j = t + k * group;
        if (has(k)) {
          if (kAgain) {
            read(k);
#pragma unroll
            for (int i = 0; i < kP; ++i) g[k][i] = g[k][i] * w[k][i];
          }
          Pair rest[kP];
          if (arrays == 3) {
            elements(stage, 2, k, rest);
#pragma unroll
            for (int i = 0; i < kP; ++i) rest[i] = RMS ? rest[i] : rest[i] + c1;
          } else {
#pragma unroll
            for (int i = 0; i < kP; ++i) rest[i] = RMS ? pair(0.f) : c1;
          }
          float f[kN];
#pragma unroll
          for (int i = 0; i < kP; ++i) {
            const float2 o = unpair(fma_pair(g[k][i], pair(inv), fma_pair(xhat[k][i], c2, rest[i])));
            f[2 * i] = o.x, f[2 * i + 1] = o.y;
          }
          row.store(to, j, V::pack(f));
        }
      }
      if (c_extra >= 0) {
        const float2 k1 = unpair(c1), k2 = unpair(c2);
        float o = fmaf(u_extra, inv, fmaf(xhat_extra, k2.x, RMS ? 0.f : k1.x));
        if (arrays == 3) o += to_float(se);
        to[c_extra] = from_float<T>(o);
      }
      to += step * p.ld_grad_x;
    }
    stage = stage == last_stage ? 0 : stage + stage_bytes;
  }

  if (p.part_w == nullptr && p.part_b == nullptr) return;
  // each group's sums go to shared memory and are added there, or, from one group, out as they are
  const int64_t part = static_cast<int64_t>(blockIdx.x) * part_ld(p.H);
  float* const part_w = p.part_w != nullptr ? p.part_w + part : nullptr;
  float* const part_b = BIAS && p.part_b != nullptr ? p.part_b + part : nullptr;
  float* to_w = part_w;
  float* to_b = part_b;
  if (groups > 1) {
    copies_arrived<0>();
    __syncthreads();
    to_w = reinterpret_cast<float*>(ring) + in_cta * row.length;
    to_b = to_w + groups * row.length;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int j = t + k * group;
    if (has(k)) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int c = row.column(j) + i;
        const float2 fw = unpair(sw[k][i / 2]), fb = unpair(sb[k][i / 2]);
        if (part_w != nullptr) to_w[c] = i % 2 ? fw.y : fw.x;
        if (part_b != nullptr) to_b[c] = i % 2 ? fb.y : fb.x;
      }
    }
  }
  if (c_extra >= 0) {
    if (part_w != nullptr) to_w[c_extra] = sw_extra;
    if (part_b != nullptr) to_b[c_extra] = sb_extra;
  }
  if (groups == 1) {
    if (LAST) add_up_here(p);
    return;
  }
  __syncthreads();
  const float* const sums = reinterpret_cast<const float*>(ring);
  for (int c = threadIdx.x; c < row.length; c += blockDim.x) {
    if (part_w != nullptr) {
      float a = 0.f;
      for (int k = 0; k < groups; ++k) a += sums[k * row.length + c];
      part_w[c] = a;
    }
    if (part_b != nullptr) {
      float a = 0.f;
      for (int k = 0; k < groups; ++k) a += sums[(groups + k) * row.length + c];
      part_b[c] = a;
    }
  }
  if (LAST) add_up_here(p);
}

// ------------------------------------------------------- any layout, by elements

// The form for rows that vectors do not fit: grad_y and x are read twice, element by
// element, which is what its time goes to.  fp32 [4096, 16384] takes 364 us (floor 121),
// bf16 [2048, 32768] 291 (60), fp16 [8191, 2047] at different places of a vector 76 (15),
// bf16 [65536, 33] 93 (2).

// The two row means of the backward pass, one CTA a row.
template <typename T, bool RMS>
__global__ void __launch_bounds__(kAnyThreads) ln_bwd_rows_any_kernel(const LnBackward p) {
  __shared__ float2 scratch[32];
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + n * p.ld_x;
    const T* g = static_cast<const T*>(p.grad_y) + n * p.ld_grad_y;
    const float mu = RMS ? 0.f : p.mean[n], inv = p.rstd[n];
    float2 a = thread_sum2(p.H, [&](int64_t h) {
      float u = to_float(g[h]);
      if (p.weight != nullptr) u *= load_elem(p.weight, p.param_dtype, h);
      return make_float2(u, u * ((to_float(x[h]) - mu) * inv));
    });
    a = block_sum2(a, scratch);
    if (threadIdx.x == 0) p.row_terms[n] = make_float2(RMS ? 0.f : a.x / p.H, a.y / p.H);
  }
}

// grad_x and the column sums, 64 columns by 4 rows a CTA at a time: CTA
// (c, s) takes columns 64 c.. and the s-th of gridDim.y ranges of rows, of which
// wide rows have few: a thread sums kBatch rows apart from those before.
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
    for (int64_t n = n0 + lane; n < n1;) {
      const int64_t end = min(n + 4 * kBatch, n1);
      float bw = 0.f, bb = 0.f;
      for (; n < end; n += 4) {
        const float mu = RMS ? 0.f : p.mean[n], inv = p.rstd[n];
        const float g = to_float(static_cast<const T*>(p.grad_y)[n * p.ld_grad_y + h]);
        const float xhat = (to_float(static_cast<const T*>(p.x)[n * p.ld_x + h]) - mu) * inv;
        bw += g * xhat;
        bb += g;
        if (p.grad_x != nullptr) {
          const float2 t = p.row_terms[n];
          float o = (g * w - t.x - xhat * t.y) * inv;
          if (p.grad_sum != nullptr) o += to_float(static_cast<const T*>(p.grad_sum)[n * p.ld_grad_sum + h]);
          static_cast<T*>(p.grad_x)[n * p.ld_grad_x + h] = from_float<T>(o);
        }
      }
      sw += bw;
      sb += bb;
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
    if (p.part_w != nullptr) p.part_w[static_cast<int64_t>(blockIdx.y) * part_ld(p.H) + h] = a.x;
    if (p.part_b != nullptr) p.part_b[static_cast<int64_t>(blockIdx.y) * part_ld(p.H) + h] = a.y;
  }
}

// Adds the partial rows of column sums in a fixed order: a CTA takes 32 columns, by
// fours, and 32 rows at a time (152 rows: all loads under way at once).  Latency is
// all it costs, 4 to 8 us.  It is launched while the kernel above still runs,
// which leaves registers enough for it to be on the SMs by then.
constexpr int kReduceThreads = 256;
__global__ void __launch_bounds__(kReduceThreads)
    ln_reduce_kernel(const float* part_w, const float* part_b, int parts, int64_t ld, int64_t H, float* grad_weight,
                     float* grad_bias, int accumulate) {
  __shared__ float scratch[kReduceThreads / 32][32];
  const bool weight = grad_weight != nullptr && blockIdx.y == 0;  // one of the two may be left out
  const float* part = weight ? part_w : part_b;
  float* out = weight ? grad_weight : grad_bias;
  const int quad = threadIdx.x & 7, warp = threadIdx.x >> 5;
  const int64_t h = static_cast<int64_t>(blockIdx.x) * 32 + quad * 4;
  grid_dependency_wait();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h < ld) {
#pragma unroll 5
    for (int k = threadIdx.x >> 3; k < parts; k += kReduceThreads / 8) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(k) * ld + h);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
  }
  if ((threadIdx.x & 31) < 8) *reinterpret_cast<float4*>(&scratch[warp][quad * 4]) = a;
  __syncthreads();
  const int64_t ho = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || ho >= H) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kReduceThreads / 32; ++k) sum += scratch[k][threadIdx.x];
  out[ho] = accumulate ? out[ho] + sum : sum;
}

// ------------------------------------------------------------------ launches

cudaError_t reduce_columns(const LnBackward& p, cudaStream_t s) {
  float *const grad_weight = p.grad_weight, *const grad_bias = p.grad_bias;
  if ((grad_weight == nullptr && grad_bias == nullptr) || p.word != nullptr) return cudaSuccess;
  prof_begin(s, FLCE_KERNEL_LN_REDUCE);
  const cudaError_t e =
      launch_after(ln_reduce_kernel,
                   dim3(static_cast<unsigned>(div_up(p.H, 32)), grad_weight != nullptr && grad_bias != nullptr ? 2 : 1),
                   dim3(kReduceThreads), s, static_cast<const float*>(p.part_w), static_cast<const float*>(p.part_b),
                   p.parts, part_ld(p.H), p.H, grad_weight, grad_bias, p.accumulate);
  prof_end(s);
  return e;
}

// Ranges of rows in the form by elements: with its strips of 64 columns, eight CTAs for each SM.
constexpr int kMostSms = 256;  // of any GPU
int64_t any_parts(int64_t H, int sms) {
  return std::min<int64_t>(div_up(int64_t(8) * std::min(sms, kMostSms), div_up(H, 64)), kMaxParts);
}

// Most vectors of a row that the vector form takes (four for each thread).
constexpr int64_t kMaxRowVectors = 2048;

// Most CTAs, and columns, whose sums a launch's last CTA adds up itself, which saves the
// host a launch where that is what a call waits for: one on [256, 128] in fp32 takes 8.3
// to 8.9 us so and 11.0 to 12.7 with a second kernel, on bf16 [512, 256] (16 CTAs) 10.2
// and 11.5 to 13.6; on bf16 [200, 1000] (25 CTAs) it would take 13.3 and takes 11.6.  (On
// the GPU alone the second kernel is 1.6 us faster.)
constexpr int64_t kMostAddedHere = 16, kMostColumnsHere = 1024;

// Most rows of a group in one launch, where column sums are wanted: a thread adds up its
// columns in one fp32 chain (3 * 2^20 equal rows of 8194 bf16 columns were off by 3e-4 of
// the sum).  More rows than that take further launches that add to the sums, of half a
// millisecond or more each: bf16 [400000, 4096] 1492 us in one, 1504 in two.
constexpr int64_t kRowsOfGroup = 1024;

constexpr size_t kSharedByDefault = 48 * 1024 - 8192;  // with the kernel's own arrays, of a CTA that asks for no more

// A launch's shape: `group` threads a row, `groups` rows a CTA, `grid` CTAs.
struct Shape {
  int group, groups;
  int64_t grid;
};

template <typename T>
Shape shape_of(const LnBackward& p, int64_t vectors, int vpt, int lanes, bool shifted) {
  constexpr int kN = Vec<T>::kN;
  Shape r;
  r.group = static_cast<int>(div_up(vectors, lanes * vpt) * lanes);
  r.groups = r.group <= 32 ? kBwdThreads / r.group : std::min(kBwdThreads / r.group, kMaxBarriers);
  r.grid = std::min<int64_t>({div_up(p.N, r.groups), device_sm_count(), kMaxParts});
  if (shifted) {  // groups a multiple of kN
    int64_t unit = kN;
    while (unit > 1 && r.groups * (unit / 2) % kN == 0) unit /= 2;
    r.grid = std::min<int64_t>(div_up(r.grid, unit), kMaxParts / unit) * unit;
  }
  return r;
}

// Lets `kernel` have `most` bytes of shared memory, once a device: the limit belongs to
// the kernel, so with each launch's own size one thread would lower it between another's
// setting it and its launch.
template <auto KERNEL>
cudaError_t allow_shared(int most) {
  static std::atomic<bool> allowed[64] = {};
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const bool kept = device >= 0 && device < 64;
  if (kept && allowed[device].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t set = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (set == cudaSuccess && kept) allowed[device].store(true, std::memory_order_release);
  return set;
}

template <typename T, bool RMS, bool BIAS, int VPT, int LANES, bool SHIFTED, bool FULL, bool LAST>
cudaError_t launch_rows(const LnBackward& p, const Shape& shape, cudaStream_t s) {
  constexpr bool kShareWeights = share_weights<T, VPT>(BIAS, SHIFTED, FULL);
  constexpr int kDepth = VPT > 2 ? 2 : kShareWeights ? 3 : 4;  // what 227 KB hold
  const int threads = shape.group * shape.groups;
  constexpr auto kernel = ln_bwd_kernel<T, RMS, BIAS, VPT, LANES, kDepth, SHIFTED, FULL, LAST>;
  // as many stages of the ring as a group has rows, and room for the groups' sums at the end
  const int64_t stages = std::min<int64_t>(kDepth, div_up(p.N, shape.grid * shape.groups));
  const int64_t slots = (p.grad_sum != nullptr ? 3 : 2) * stages + (kShareWeights ? 2 : 0);
  const int64_t sums = shape.groups > 1 ? shape.groups * p.H * 4 * 2 : 0;
  const size_t smem = static_cast<size_t>(std::max<int64_t>(int64_t(threads) * VPT * 16 * slots, sums));
  if (smem > kSharedByDefault) {
    // the whole ring: 96 bytes or more for each of a CTA's vectors, of which the groups' sums take at most 64 (and
    // for what lies beside shifted ones a little more)
    constexpr int kMost = kBwdThreads * VPT * 16 * (3 * kDepth + (kShareWeights ? 2 : 0));
    if (smem > kMost) return cudaErrorInvalidConfiguration;
    const cudaError_t e = allow_shared<kernel>(kMost);
    if (e != cudaSuccess) return e;
  }
  kernel<<<static_cast<unsigned int>(shape.grid), threads, smem, s>>>(p, shape.group, shape.groups);
  return cudaGetLastError();
}

// Launches the first rows of p (as many as one launch takes: p.N after it).
template <typename T, bool RMS, bool BIAS, int VPT, int LANES, bool SHIFTED>
cudaError_t backward_rows(LnBackward& p, int64_t vectors, cudaStream_t s) {
  const Shape shape = shape_of<T>(p, vectors, VPT, LANES, SHIFTED);
  // a multiple of 1024, so that the next launch's first row starts at the same place of a vector
  if (p.part_w != nullptr || p.part_b != nullptr)
    p.N = std::min(p.N, kRowsOfGroup * shape.grid * shape.groups);
  p.parts = static_cast<int>(shape.grid);
  if constexpr (VPT <= 2) {
    if (p.word != nullptr && shape.grid <= kMostAddedHere && p.H <= kMostColumnsHere)
      return launch_rows<T, RMS, true, VPT, LANES, SHIFTED, false, true>(p, shape, s);
  }
  p.word = nullptr;
  if constexpr (!SHIFTED) {
    if (vectors == static_cast<int64_t>(shape.group) * VPT)
      return launch_rows<T, RMS, BIAS, VPT, LANES, SHIFTED, true, false>(p, shape, s);
  }
  return launch_rows<T, RMS, BIAS, VPT, LANES, SHIFTED, false, false>(p, shape, s);
}

// Two vectors a thread; four where 512 threads hold no row otherwise; and, where rows
// start inside a vector, one if a warp's threads are enough then (it takes a whole warp
// for the columns beside the vectors).  Of a warp, 16 or 8 lanes take a row that fills
// no more: [65536, 128] in fp32 28.6 -> 23.4 us, in bf16 26.8 -> 20.5, bf16 [65536, 256]
// 30.2 -> 27.5, all against a warp with one vector a lane.
template <typename T, bool RMS, bool BIAS, bool SHIFTED>
cudaError_t backward_rows(LnBackward& p, int64_t vectors, cudaStream_t s) {
  if constexpr (SHIFTED) {
    if (vectors <= 32) return backward_rows<T, RMS, BIAS, 1, 32, SHIFTED>(p, vectors, s);
  } else {
    if (vectors <= 16) return backward_rows<T, RMS, BIAS, 2, 8, SHIFTED>(p, vectors, s);
    if (vectors <= 32) return backward_rows<T, RMS, BIAS, 2, 16, SHIFTED>(p, vectors, s);
  }
  if (vectors <= 2 * kBwdThreads) return backward_rows<T, RMS, BIAS, 2, 32, SHIFTED>(p, vectors, s);
  return backward_rows<T, RMS, BIAS, 4, 32, SHIFTED>(p, vectors, s);
}

// The call's rows from n on, which add to the sums of those before.
template <typename T>
LnBackward rows_from(LnBackward p, int64_t n) {
  const auto at = [n](const void* m, int64_t ld) { return m != nullptr ? static_cast<const T*>(m) + n * ld : nullptr; };
  p.grad_y = at(p.grad_y, p.ld_grad_y);
  p.x = at(p.x, p.ld_x);
  p.grad_sum = at(p.grad_sum, p.ld_grad_sum);
  if (p.grad_x != nullptr) p.grad_x = static_cast<T*>(p.grad_x) + n * p.ld_grad_x;
  if (p.mean != nullptr) p.mean += n;
  p.rstd += n;
  p.N -= n;
  if (n > 0) p.accumulate = 1;
  return p;
}

template <typename T, bool RMS>
cudaError_t backward(LnBackward p, cudaStream_t s) {
  p.parts = 0;
  if (p.N == 0) p.word = nullptr;
  const Fit fit = fit_of<T>(p.N, p.H, p.weight, nullptr, p.param_dtype, Matrix{p.x, p.ld_x},
                            Matrix{p.grad_y, p.ld_grad_y}, Matrix{p.grad_sum, p.ld_grad_sum},
                            Matrix{p.grad_x, p.ld_grad_x});
  const int64_t vectors = p.H / Vec<T>::kN;  // where rows start inside one, a few less
  cudaError_t e = cudaSuccess;
  if (p.N > 0 && fit != kFitNot && vectors <= kMaxRowVectors) {
    for (int64_t n = 0; n < p.N;) {
      LnBackward q = rows_from<T>(p, n);
      prof_begin(s, FLCE_KERNEL_LN_BWD);
      // a bias is rare without a mean and usual with one: without a mean it has a form of its own
      if (RMS && p.part_b == nullptr)
        e = fit == kFitWhole ? backward_rows<T, RMS, !RMS, false>(q, vectors, s)
                             : backward_rows<T, RMS, !RMS, true>(q, vectors, s);
      else
        e = fit == kFitWhole ? backward_rows<T, RMS, true, false>(q, vectors, s)
                             : backward_rows<T, RMS, true, true>(q, vectors, s);
      prof_end(s);
      if (e == cudaSuccess) e = reduce_columns(q, s);
      if (e != cudaSuccess) return e;
      n += q.N;
    }
    return cudaSuccess;
  } else if (p.N > 0) {
    p.word = nullptr;
    const int sms = device_sm_count();
    if (p.grad_x != nullptr) {
      prof_begin(s, FLCE_KERNEL_LN_BWD);
      ln_bwd_rows_any_kernel<T, RMS>
          <<<static_cast<int>(std::min<int64_t>(p.N, int64_t(8) * sms)), kAnyThreads, 0, s>>>(p);
      e = cudaGetLastError();
      prof_end(s);
      if (e != cudaSuccess) return e;
    }
    const int64_t strips = div_up(p.H, 64);
    p.parts = static_cast<int>(std::min<int64_t>(any_parts(p.H, sms), div_up(p.N, 4)));
    prof_begin(s, FLCE_KERNEL_LN_BWD);
    ln_bwd_cols_any_kernel<T, RMS><<<dim3(static_cast<unsigned>(strips), p.parts), kAnyThreads, 0, s>>>(p);
    e = cudaGetLastError();
    prof_end(s);
    if (e != cudaSuccess) return e;
  }
  return reduce_columns(p, s);
}

struct LnLayout {
  size_t row_terms, part_w, part_b, word, total;
};

LnLayout ln_layout(int64_t N, int64_t H) {
  LnLayout L;
  // a partial row of sums for each CTA: at most one a row, rounded up to eight (the places in a vector where rows
  // start); rows too long for vectors take ranges of rows by strips of columns, few of them
  const int64_t most = H / 8 <= kMaxRowVectors ? kMaxParts : any_parts(H, kMostSms);
  const int64_t parts = std::min<int64_t>(div_up(std::max<int64_t>(N, 1), 8) * 8, most);
  const size_t part = align_up(static_cast<size_t>(parts) * part_ld(H) * 4, 256);
  L.row_terms = 0;
  L.part_w = align_up(static_cast<size_t>(N) * sizeof(float2), 256);
  L.part_b = L.part_w + part;
  L.word = L.part_b + part;
  L.total = L.word + 256;
  return L;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

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
  const bool sums = grad_weight != nullptr || grad_bias != nullptr;
  LnBackward p = {grad_y,
                  x,
                  weight,
                  grad_sum,
                  mean,
                  rstd,
                  grad_x,
                  ld_grad_y,
                  ld_x,
                  ld_grad_sum,
                  ld_grad_x,
                  N,
                  H,
                  param_dtype,
                  reinterpret_cast<float2*>(ws + L.row_terms),
                  grad_weight != nullptr ? reinterpret_cast<float*>(ws + L.part_w) : nullptr,
                  grad_bias != nullptr ? reinterpret_cast<float*>(ws + L.part_b) : nullptr,
                  0,
                  grad_weight,
                  grad_bias,
                  accumulate,
                  sums ? reinterpret_cast<unsigned long long*>(ws + L.word) : nullptr,
                  next_arrival_tag()};
  return LN_BY_TYPE(backward, p, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
