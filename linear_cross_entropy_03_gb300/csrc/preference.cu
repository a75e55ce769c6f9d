// The loss over pairs of sequences by their log-probability ratios to a reference model,
// and its gradient on the logits.  A pair's loss needs every row of both sequences before
// its first gradient, so this takes three launches: row statistics (M, S and logp of each
// row: row_loss.cuh), the pairs, and the rows' gradients
//     grad = f (p - onehot(t)),   f = -slope * (+1 chosen, -1 rejected) [/ tokens]
// with slope the loss's by x.  The logits are read twice: 3 N V elements move, less what
// the second reading finds in L2, where the last rows of the first one still are, as it
// runs from the last row to the first.
#include "row_loss.cuh"

namespace flce {
namespace {

struct PairParams {
  const int64_t* target;
  const int64_t* offsets;  // or null: sequences of `length` rows
  int64_t length;
  const float* ref_logp;
  const float* grad_out;
  const float* logp_rows;  // [N]
  int64_t N, V, pairs, ignore_index;
  flce_preference_t numbers;
  int reduction;
  double scale;        // grad_scale, or that over the pairs of a mean
  float* factor;       // [N]
  double* pair_loss;   // [pairs]
  float* loss;
  float* logp;
  int* status;
  int add_up;          // whether the losses are added up here (else by the gradients' launch)
  unsigned long long* arrivals;
  unsigned long long tag;
};

constexpr int kPairThreads = 256;

// Rows of a sequence, cut to [0, N).
__device__ __forceinline__ void sequence_rows(const PairParams& p, int64_t q, int64_t* from, int64_t* to, int* bits) {
  int64_t a = q * p.length, b = a + p.length;
  if (p.offsets != nullptr) {
    a = __ldg(p.offsets + q), b = __ldg(p.offsets + q + 1);
    if (a < 0 || b < a || b > p.N) *bits |= FLCE_STATUS_BIT_SEQUENCE_RANGE;
    a = a < 0 ? 0 : a > p.N ? p.N : a;
    b = b < a ? a : b > p.N ? p.N : b;
  }
  *from = a, *to = b;
}

// The sum over the threads of each half of the CTA, for thread 0 of the half; by its first
// warp, as an SM has two fp64 operations a cycle.
__device__ __forceinline__ double half_sum(double v, double* scratch) {
  scratch[threadIdx.x] = v;
  __syncthreads();
  double total = 0;
  const int t = threadIdx.x % (kPairThreads / 2);
  if (t < 32) {
#pragma unroll
    for (int i = 0; i < kPairThreads / 2; i += 32) total += scratch[threadIdx.x + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  __syncthreads();
  return total;
}

// The loss of SUM and MEAN, by a CTA's first warp, in an order that the number of pairs fixes.
__device__ __forceinline__ void add_up_losses(const double* pair_loss, int64_t pairs, int reduction, float* loss) {
  if (threadIdx.x >= 32) return;
  double total = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < pairs; i += 32) total += __ldcg(pair_loss + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (threadIdx.x == 0)
    *loss = static_cast<float>(reduction == FLCE_REDUCTION_MEAN ? total / static_cast<double>(pairs) : total);
}

// One CTA a pair, half of it for each sequence.  Sums are fp64 in an order that the lengths
// fix.
__global__ void __launch_bounds__(kPairThreads) pair_loss_kernel(const PairParams p) {
  constexpr int kHalf = kPairThreads / 2;
  __shared__ double scratch[kPairThreads];
  __shared__ double sums[2], tokens_of[2], slope_of_pair;
  __shared__ int last, all_bits;
  const int half = threadIdx.x / kHalf, t = threadIdx.x % kHalf;
  if (threadIdx.x == 0) {
    all_bits = 0;
    if (blockIdx.x == 0 && p.add_up) expect_arrivals(p.arrivals, p.tag);
  }
  __syncthreads();
  grid_dependency_wait();
  int bits = 0;
  for (int64_t pair = blockIdx.x; pair < p.pairs; pair += gridDim.x) {
    int64_t from, to;
    sequence_rows(p, pair + half * p.pairs, &from, &to, &bits);
    const float ref[2] = {p.ref_logp != nullptr ? __ldg(p.ref_logp + pair) : 0.f,
                          p.ref_logp != nullptr ? __ldg(p.ref_logp + pair + p.pairs) : 0.f};
    double sum = 0;
    int64_t tokens = 0;
#pragma unroll 4
    for (int64_t n = from + t; n < to; n += kHalf) {
      const int64_t target = __ldg(p.target + n);
      const float logp = p.logp_rows[n];
      if (target == p.ignore_index || target < 0 || target >= p.V) continue;
      sum += static_cast<double>(logp);
      ++tokens;
    }
    sum = half_sum(sum, scratch);
    double count = 1;
    if (p.numbers.average) {
      count = half_sum(static_cast<double>(tokens), scratch);
      if (t == 0 && count > 1) sum /= count;
      if (count < 1) count = 1;
    }
    if (t == 0) sums[half] = sum, tokens_of[half] = count;
    __syncthreads();
    const double s[2] = {sums[0], sums[1]};
    if (threadIdx.x == 0) {
      // differences of long sums in fp64, functions of the difference in fp32
      double x = s[0] - s[1];
      x -= static_cast<double>(ref[0]) - ref[1];
      const double beta = p.numbers.beta;
      double loss, slope;  // slope: dloss / dx
      if (p.numbers.kind == FLCE_PREFERENCE_IPO) {
        const double far = x - 1.0 / (2.0 * beta);
        loss = far * far;
        slope = 2.0 * far;
      } else {
        const double wide = beta * x - p.numbers.margin;
        const float u = static_cast<float>(wide);
        if (p.numbers.kind == FLCE_PREFERENCE_HINGE) {
          loss = wide < 1.0 ? 1.0 - wide : wide >= 1.0 ? 0.0 : wide;  // (NaN stays)
          slope = wide < 1.0 ? -beta : wide >= 1.0 ? 0.0 : wide;
        } else {
          // ln sigmoid(-u) = ln sigmoid(u) - u
          const float e = expf(-fabsf(u)), smooth = p.numbers.label_smoothing;
          loss = fmax(-wide, 0.0) + log1pf(e) + (smooth != 0.f ? smooth * wide : 0.0);  // (u may be infinite)
          if (isnan(u)) loss = wide;
          const float less = u >= 0.f ? e / (1.f + e) : 1.f / (1.f + e);  // 1 - sigmoid(u)
          slope = beta * (static_cast<double>(smooth) - less);
        }
      }
      slope_of_pair = slope * p.scale * (p.grad_out != nullptr ? p.grad_out[pair] : 1.f);
      p.pair_loss[pair] = loss;
      if (p.reduction == FLCE_REDUCTION_NONE) p.loss[pair] = static_cast<float>(loss);
      if (p.logp != nullptr) {
        p.logp[pair] = static_cast<float>(s[0]);
        p.logp[pair + p.pairs] = static_cast<float>(s[1]);
      }
    }
    __syncthreads();
    float f = 0.f;
    if (t % 32 == 0) {
      const double slope = half == 0 ? -slope_of_pair : slope_of_pair;
      f = static_cast<float>(p.numbers.average ? slope / tokens_of[half] : slope);
    }
    f = __shfl_sync(0xffffffffu, f, 0);
    for (int64_t n = from + t; n < to; n += kHalf) p.factor[n] = f;
    __syncthreads();  // the sums are the next pair's
  }
  if (bits != 0) atomicOr(&all_bits, bits);
  __syncthreads();
  if (threadIdx.x == 0) {
    if (all_bits != 0) atomicOr(p.status, all_bits);
    last = p.add_up && arrives_last(p.arrivals, p.tag, gridDim.x);
  }
  __syncthreads();
  if (last) add_up_losses(p.pair_loss, p.pairs, p.reduction, p.loss);
}

struct GradParams {
  const void* logits;
  void* grad;
  int64_t ld, ld_grad, N, V, ignore_index;
  const int64_t* target;
  const float2* stats;   // (M, 1 / S) of each row
  const float* factor;   // f of each row
  const float* logp;
  int64_t parts;         // pieces of a row
  int64_t items;         // rows times parts
  const double* pair_loss;
  int64_t pairs;
  int reduction;
  float* loss;           // of SUM and MEAN: by the first CTA
};

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;

// A piece of a row by each CTA (or by each warp, where a row is short), from the last row
// to the first, so that it meets in L2 what the statistics read last.  Bound by memory: bf16
// [2985, 128256] 213 us, 7.2 TB/s of reading and writing.
template <typename T, int GROUP>
__global__ void __launch_bounds__(kGradThreads) row_grad_kernel(const GradParams p) {
  constexpr int kE = kVecElems<T>;
  const int lane = threadIdx.x % GROUP;
  if (blockIdx.x == 0) {
    grid_dependency_wait();
    if (p.reduction != FLCE_REDUCTION_NONE) add_up_losses(p.pair_loss, p.pairs, p.reduction, p.loss);
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x - 1) * (kGradThreads / GROUP) + threadIdx.x / GROUP;
  if (item >= p.items) return;
  const int64_t row = p.N - 1 - item / p.parts, part = item % p.parts;
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  T* g = static_cast<T*>(p.grad) + row * p.ld_grad;
  const RowSplit split = split_row(x, p.V);
  const bool vector = same_phase(x, g);
  const uint4* vecs = reinterpret_cast<const uint4*>(x + split.head);
  uint4 v[kGradVecs];
  const int64_t first = part * (GROUP * kGradVecs) + lane;
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i)
    if (first + i * GROUP < split.vecs) v[i] = vecs[first + i * GROUP];
  // one element before or after the vectors: by the lanes of the first and the last piece
  int64_t extra = -1;
  if (part == 0 && lane < split.head) extra = lane;
  if (part == p.parts - 1 && lane >= 8 && lane < 8 + split.tail) extra = split.head + split.vecs * kE + lane - 8;
  const float z = extra >= 0 ? to_float(x[extra]) : 0.f;
  const int64_t target = __ldg(p.target + row);
  grid_dependency_wait();
  const float2 stats = p.stats[row];
  float f = p.factor[row];
  const bool live = target != p.ignore_index && target >= 0 && target < p.V;
  const bool zero = !live || f == 0.f;
  const Pair minus_m = pair(-stats.x), c = pair(kLog2E), factor = pair(f * stats.y);
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int64_t at = first + i * GROUP;
    if (at >= split.vecs) break;
    const uint4 out = zero ? make_uint4(0, 0, 0, 0) : vec_grad<T>(v[i], minus_m, c, factor);
    store_vec<T>(g + split.head + at * kE, out, vector);
  }
  if (extra >= 0) g[extra] = from_float<T>(zero ? 0.f : f * stats.y * ex2_approx((z - stats.x) * kLog2E));
  if (zero) return;
  // the target's element, by the thread that wrote it
  bool mine = extra == target;
  const int64_t inside = target - split.head;
  if (inside >= 0 && inside < split.vecs * kE) {
    const int64_t at = inside / kE - part * (GROUP * kGradVecs);
    mine = at >= 0 && at < GROUP * kGradVecs && at % GROUP == lane;
  }
  if (mine) g[target] = from_float<T>(f * expm1f(p.logp[row]));
}

template <typename T>
cudaError_t launch_grad(GradParams p, cudaStream_t s) {
  const int64_t vecs = p.V / kVecElems<T>;
  const bool by_warps = vecs <= 32 * kGradVecs;
  p.parts = vecs < 1 ? 1 : div_up(vecs, (by_warps ? 32 : kGradThreads) * kGradVecs);
  p.items = p.N * p.parts;
  const int64_t ctas = 1 + (by_warps ? div_up(p.items, kGradThreads / 32) : p.items);
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  return by_warps ? launch_after(row_grad_kernel<T, 32>, grid, dim3(kGradThreads), s, p)
                  : launch_after(row_grad_kernel<T, kGradThreads>, grid, dim3(kGradThreads), s, p);
}

// Workspace after the part that all row losses have: logp, factors and (M, 1 / S) of the
// rows, and the pairs' losses.
struct PreferenceLayout {
  size_t logp, factor, stats, pairs, total;
};

bool preference_layout(int64_t N, int64_t pairs, PreferenceLayout* at) {
  if (N < 0 || N >= (int64_t(1) << 31) || pairs < 0 || pairs >= (int64_t(1) << 30)) return false;
  at->logp = align_up(kRowLossFixed, 256);
  at->factor = align_up(at->logp + N * 4, 256);
  at->stats = align_up(at->factor + N * 4, 256);
  at->pairs = align_up(at->stats + N * 8, 256);
  at->total = align_up(at->pairs + pairs * 8, 256);
  return true;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

size_t preference_workspace_size(int64_t N, int64_t pairs) {
  PreferenceLayout at;
  return preference_layout(N, pairs, &at) ? at.total : 0;
}

flce_status_t preference_fwd_bwd(const void* logits, int dtype, int64_t ld, void* grad_logits, int64_t ld_grad,
                                 const int64_t* target, const int64_t* offsets, const float* ref_logp, int64_t pairs,
                                 int64_t N, int64_t V, const flce_preference_t* numbers, int64_t ignore_index,
                                 int reduction, float grad_scale, const float* grad_out_none, float* loss, float* logp,
                                 void* workspace, size_t workspace_bytes, int32_t* status_dev,
                                 flce_stream_t stream_) {
  PreferenceLayout at;
  if (!preference_layout(N, pairs, &at)) return FLCE_ERR_INVALID_ARG;
  const flce_status_t st = check_rows(logits, dtype, ld, grad_logits, ld_grad, N, V, pairs, reduction, grad_out_none,
                                      loss, workspace, workspace_bytes, at.total, status_dev);
  if (st != FLCE_OK) return st;
  if (numbers == nullptr || (N > 0 && target == nullptr)) return FLCE_ERR_INVALID_ARG;
  const int kind = numbers->kind;
  if (kind < FLCE_PREFERENCE_SIGMOID || kind > FLCE_PREFERENCE_IPO || (numbers->average & ~1) != 0 ||
      !positive(numbers->beta) || !(numbers->label_smoothing >= 0.f && numbers->label_smoothing < 1.f) ||
      !(numbers->margin - numbers->margin == 0.f))
    return FLCE_ERR_INVALID_ARG;
  if ((numbers->label_smoothing != 0.f && kind != FLCE_PREFERENCE_SIGMOID) ||
      (numbers->margin != 0.f && kind == FLCE_PREFERENCE_IPO))
    return FLCE_ERR_INVALID_ARG;
  if (offsets == nullptr && (pairs == 0 ? N != 0 : N % (2 * pairs) != 0)) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(target, 8) || !aligned_to(offsets, 8) || !aligned_to(ref_logp, 4) || !aligned_to(logp, 4))
    return FLCE_ERR_MISALIGNED;
  // the pieces of all rows are one launch's CTAs
  if (grad_logits != nullptr && N * div_up(V, 1024) >= (int64_t(1) << 31)) return FLCE_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  RowLossParams p = row_params(logits, ld, nullptr, ld, N, V, FLCE_REDUCTION_SUM, 1.f, nullptr, nullptr, 1.f);
  p.loss_rows = p.loss = nullptr;
  p.ignore_index = ignore_index, p.target = target;
  p.logp = reinterpret_cast<float*>(ws + at.logp);
  p.factor = reinterpret_cast<float*>(ws + at.factor);
  p.stats = reinterpret_cast<float2*>(ws + at.stats);
  use_workspace(&p, workspace, status_dev);
  if (launch_rows<kStats>(p, dtype, stream) != cudaSuccess) return FLCE_ERR_CUDA;

  PairParams q = {};
  q.target = target, q.offsets = offsets, q.length = pairs > 0 ? N / (2 * pairs) : 0;
  q.ref_logp = ref_logp, q.grad_out = grad_out_none, q.logp_rows = p.logp;
  q.N = N, q.V = V, q.pairs = pairs, q.ignore_index = ignore_index, q.numbers = *numbers;
  q.reduction = reduction, q.factor = p.factor;
  q.scale = reduction == FLCE_REDUCTION_MEAN && pairs > 0 ? grad_scale / static_cast<double>(pairs) : grad_scale;
  q.pair_loss = reinterpret_cast<double*>(ws + at.pairs);
  q.loss = loss, q.logp = logp, q.status = p.status;
  const bool grads = grad_logits != nullptr && N > 0;
  q.add_up = reduction != FLCE_REDUCTION_NONE && !grads;
  q.arrivals = p.arrivals + 1, q.tag = next_arrival_tag();
  const int64_t most = 8 * device_sm_count();
  prof_begin(stream, FLCE_KERNEL_PAIR_LOSS);
  cudaError_t e = launch_after(pair_loss_kernel, dim3(static_cast<unsigned>(pairs < 1 ? 1 : pairs < most ? pairs : most)),
                               dim3(kPairThreads), stream, q);
  prof_end(stream);
  if (e != cudaSuccess) return FLCE_ERR_CUDA;
  if (!grads) return FLCE_OK;

  const GradParams g = {logits, grad_logits, ld, ld_grad, N,     V,         ignore_index, target, p.stats, p.factor,
                        p.logp, 0,           0,  q.pair_loss, pairs, reduction, loss};
  prof_begin(stream, FLCE_KERNEL_ROW_GRAD);
  e = dtype == FLCE_DTYPE_BF16   ? launch_grad<__nv_bfloat16>(g, stream)
      : dtype == FLCE_DTYPE_FP16 ? launch_grad<__half>(g, stream)
                                 : launch_grad<float>(g, stream);
  prof_end(stream);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
