// Losses on materialised logits [N, V] that a row's softmax and a few numbers of its own
// give: the clipped policy loss, the distance from a teacher's top logits, and the row
// statistics of the preference loss.  With z the row's logits, T the temperature,
// M = max z, S = sum exp((z - M) / T) and p = exp((z - M) / T) / S:
//
//   policy      logp = (z_t - M) / T - ln S, r = exp(logp - old), d = ref - logp
//               loss = -min(r A, clip(r) A) + b (exp(d) - 1 - d)
//               slope = dloss / dlogp = -r A [not clipped] - b (exp(d) - 1)
//               grad = f (p - onehot(t)),  f = -slope / T
//   distill     q = softmax of the teacher's values / T,
//               loss = T^2 sum_k q_k (ln q_k - ln p_k),  grad = f (p - q),  f = T
//
// so a row is read, reduced to (M, S) and written as f p, but for the few places that the
// target or the teacher's list names.  Everything between loading and storing is fp32,
// sums over rows are fp64.  Logits about any common level keep their digits: differences
// z - M are formed before they are scaled (rows by warps, rows that are read twice), or in
// the operation that scales (rows by parts, below kFarExponent).
#pragma once

#include <atomic>
#include <cfloat>
#include <type_traits>

#include "arrival.cuh"
#include "elem.cuh"
#include "ptx.cuh"

namespace flce {

constexpr int kMaxTeacher = 1024;      // entries of a teacher's list
constexpr int kRowLossMaxCtas = 4096;  // partial losses in the workspace
constexpr int kCountCtas = 64;         // partial counts of the rows that take part

// kDistill: lists of up to 64 entries; kDistillLong: any.
enum RowLoss { kPolicy = 0, kDistill = 1, kStats = 2, kDistillLong = 3 };
constexpr bool has_list(int kind) { return kind == kDistill || kind == kDistillLong; }

struct RowLossParams {
  const void* logits;
  void* grad;  // may be logits; null: loss only
  int64_t ld, ld_grad;
  int64_t N, V;
  int64_t ignore_index;
  const int64_t* target;  // policy, stats
  const float* advantage;
  const float* old_logp;  // or null
  const float* ref_logp;  // or null
  float ratio_low, ratio_high, kl_weight;
  const void* ids;  // distill: [N, K]
  const void* values;
  int ids32, value_dtype, K;
  const float* row_weight;  // [N] or null
  const float* grad_out;    // [N] or null
  float temperature, inv_t, c;  // T, 1 / T, log2(e) / T
  int reduction;
  float grad_scale;
  float* loss_rows;  // reduction none, else null
  float* loss;       // sum and mean, else null
  float* logp;       // [N] or null
  float2* stats;     // stats: (M, 1 / S) of each row
  float* factor;     // stats: [N], set to 0
  // workspace
  const int* counts;  // kCountCtas partial counts, or null: the kernel counts itself
  double* partial;    // [grid]
  int* flags;         // [grid]
  unsigned long long* arrivals;
  unsigned long long tag;
  int* status;
  int own_status;  // the workspace's own word: written, and not added to
  uint64_t timeout_ns;
};

namespace {

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ int64_t load_id(const void* ids, int ids32, int64_t i) {
  return ids32 ? __ldg(static_cast<const int32_t*>(ids) + i) : __ldg(static_cast<const int64_t*>(ids) + i);
}

// ---------------------------------------------------------------- vectors of a row

// Eight 16-bit elements or four of fp32.
template <typename T>
constexpr int kVecElems = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ void vec_pairs(const uint4& v, Pair (&to)[kVecElems<T> / 2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
    to[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
    to[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(reinterpret_cast<const __half2&>(w[k]));
        to[k] = pair(f.x, f.y);
      } else {
        to[k] = pair(bf16_lo(w[k]), bf16_hi(w[k]));
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const Pair (&from)[kVecElems<T> / 2]) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
    const float2 a = unpair(from[0]), b = unpair(from[1]);
    w[0] = __float_as_uint(a.x), w[1] = __float_as_uint(a.y), w[2] = __float_as_uint(b.x), w[3] = __float_as_uint(b.y);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpair(from[k]);
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        w[k] = reinterpret_cast<const uint32_t&>(h);
      } else {
        w[k] = pack_bf16x2(f.x, f.y);
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A vector that adds nothing to a row.
template <typename T>
__device__ __forceinline__ uint4 empty_vec() {
  const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
  return make_uint4(w, w, w, w);
}

// The largest element; NaN is passed over here (the sum of exponentials shows it).
template <typename T, int COUNT>
__device__ __forceinline__ float vecs_max(const uint4 (&v)[COUNT]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y))),
                fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w)));
    return m;
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 m = reinterpret_cast<const T2&>(v[0].x);
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const T2* w = reinterpret_cast<const T2*>(&v[i]);
      m = __hmax2(m, __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
    }
    return fmaxf(__low2float(m), __high2float(m));
  }
}

// exp((z - M) / T) of a vector's elements, with c = log2(e) / T.
template <typename T>
__device__ __forceinline__ void vec_exp(const uint4& v, Pair minus_m, Pair c, Pair (&e)[kVecElems<T> / 2]) {
  vec_pairs<T>(v, e);
#pragma unroll
  for (int k = 0; k < kVecElems<T> / 2; ++k) {
    const float2 x = unpair((e[k] + minus_m) * c);
    e[k] = pair(ex2_approx(x.x), ex2_approx(x.y));
  }
}

template <typename T>
__device__ __forceinline__ void vec_add_exp(const uint4& v, Pair minus_m, Pair c, Pair& sum) {
  Pair e[kVecElems<T> / 2];
  vec_exp<T>(v, minus_m, c, e);
#pragma unroll
  for (int k = 0; k < kVecElems<T> / 2; ++k) sum = sum + e[k];
}

// Elements factor * exp((z - M) / T): a row's gradient but for the places that it names.
template <typename T>
__device__ __forceinline__ uint4 vec_grad(const uint4& v, Pair minus_m, Pair c, Pair factor) {
  Pair e[kVecElems<T> / 2];
  vec_exp<T>(v, minus_m, c, e);
#pragma unroll
  for (int k = 0; k < kVecElems<T> / 2; ++k) e[k] = e[k] * factor;
  return pack_pairs<T>(e);
}

// A vector of a gradient's row, of which `vector` says whether it lies on a boundary there.
template <typename T>
__device__ __forceinline__ void store_vec(T* to, const uint4& v, bool vector) {
  if (vector) {
    __stcs(reinterpret_cast<uint4*>(to), v);
  } else {
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int k = 0; k < kVecElems<T>; ++k) to[k] = e[k];
  }
}

// A row's elements: `head` before the first 16-byte boundary, `vecs` vectors, `tail` after.
struct RowSplit {
  int head, tail, vecs;
};

template <typename T>
__device__ __forceinline__ RowSplit split_row(const T* row, int64_t V) {
  constexpr unsigned kE = kVecElems<T>;
  const unsigned v = static_cast<unsigned>(V);  // (below 2^31)
  const unsigned place = (16u - (static_cast<unsigned>(reinterpret_cast<uintptr_t>(row)) & 15u)) & 15u;
  const unsigned head = min(place / static_cast<unsigned>(sizeof(T)), v);
  RowSplit s;
  s.head = static_cast<int>(head);
  s.vecs = static_cast<int>((v - head) / kE);
  s.tail = static_cast<int>((v - head) % kE);
  return s;
}

// Whether vectors of a row of logits lie on boundaries of the gradient's row too.
template <typename T>
__device__ __forceinline__ bool same_phase(const T* x, const T* g) {
  return ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(g)) & 15) == 0;
}

// Partial results (m, s) of parts of a row, as (M, S): by all lanes, each with one part
// (or several combined before), parts of nothing as (-inf, 0).
__device__ __forceinline__ float2 combine_parts(float m, float s, float c) {
  const float top = warp_max_redux(m);
  const float shift = top > -INFINITY ? top : 0.f;
  return make_float2(top, warp_sum(m > -INFINITY ? s * ex2_approx((m - shift) * c) : s));
}

// ---------------------------------------------------------------- what a row has beside its logits

struct RowInfo {
  float zt;  // policy, stats: the target's logit; distill: the largest logit of the list
  float advantage, old_logp, ref_logp;
  float weight, grad_out;
  float a;      // distill: sum of q (ln q - (z - zt) / T)
  int column;   // policy, stats: the target's, or -1 where the row takes no part
  bool taught;  // distill: whether the row has a teacher
  int entries;  // distill: length of the list
};

// What a row has beside its logits is read in two steps, as the second (logits at places that
// the first names) needs the first: a warp that leads others starts both ahead of the row,
// and looks at what it has read when it comes to the row (what is read stays as it lies in
// memory until then: a conversion would wait for it).  Rows past the end have nothing.
template <typename T>
struct Raw {
  T v;
};
template <>
struct Raw<__half> {
  uint16_t v;
};
template <>
struct Raw<__nv_bfloat16> {
  uint16_t v;
};
template <typename T>
__device__ __forceinline__ Raw<T> raw_logit(const RowLossParams& p, int64_t row, int64_t column) {
  return reinterpret_cast<const Raw<T>*>(p.logits)[row * p.ld + column];
}
template <typename T>
__device__ __forceinline__ float raw_float(Raw<T> r) {
  if constexpr (sizeof(T) == 4)
    return r.v;
  else if constexpr (std::is_same<T, __half>::value)
    return __half2float(__ushort_as_half(r.v));
  else
    return __uint_as_float(static_cast<uint32_t>(r.v) << 16);
}

template <typename T>
struct PolicyAhead {
  int64_t target;
  float weight, grad_out, advantage, old_logp, ref_logp;
  Raw<T> z;
};
template <typename T>
__device__ __forceinline__ PolicyAhead<T> policy_ahead(const RowLossParams& p, int64_t row) {
  PolicyAhead<T> a = {};
  a.target = p.ignore_index;
  a.weight = a.grad_out = 1.f;
  if (row >= p.N) return a;
  a.target = __ldg(p.target + row);
  if (p.row_weight != nullptr) a.weight = __ldg(p.row_weight + row);
  if (p.grad_out != nullptr) a.grad_out = __ldg(p.grad_out + row);
  if (p.advantage != nullptr) a.advantage = __ldg(p.advantage + row);
  if (p.old_logp != nullptr) a.old_logp = __ldg(p.old_logp + row);
  if (p.ref_logp != nullptr) a.ref_logp = __ldg(p.ref_logp + row);
  return a;
}
template <typename T>
__device__ __forceinline__ void policy_logit(const RowLossParams& p, int64_t row, PolicyAhead<T>& a) {
  if (a.target != p.ignore_index && a.target >= 0 && a.target < p.V) a.z = raw_logit<T>(p, row, a.target);
}
template <typename T>
__device__ __forceinline__ RowInfo policy_info(const RowLossParams& p, const PolicyAhead<T>& a, int* bits) {
  RowInfo r = {};
  r.weight = a.weight, r.grad_out = a.grad_out, r.advantage = a.advantage;
  r.old_logp = a.old_logp, r.ref_logp = a.ref_logp;
  r.column = -1;
  if (a.target == p.ignore_index) return r;
  if (a.target < 0 || a.target >= p.V) {
    *bits |= FLCE_STATUS_BIT_TARGET_RANGE;
    return r;
  }
  r.column = static_cast<int>(a.target);
  r.zt = raw_float<T>(a.z);
  return r;
}
template <typename T>
__device__ __forceinline__ RowInfo policy_row(const RowLossParams& p, int64_t row, int* bits) {
  PolicyAhead<T> a = policy_ahead<T>(p, row);
  policy_logit<T>(p, row, a);
  return policy_info<T>(p, a, bits);
}

// A teacher's list in shared memory: columns (-1: no such place), shares and logits.
struct TeacherList {
  int* column;
  float* q;
  float* z;
};
__host__ __device__ constexpr int list_room(int K) { return (K + 31) & ~31; }
__host__ __device__ constexpr size_t list_bytes(int K) { return static_cast<size_t>(list_room(K)) * 12; }
// Slots of the table that finds columns that a list names twice: at least twice the entries.
__host__ __device__ constexpr int table_slots(int K) {
  int n = 64;
  while (n < 2 * K) n *= 2;
  return n;
}
__device__ __forceinline__ TeacherList list_at(uint8_t* at, int K) {
  const int room = list_room(K);
  return {reinterpret_cast<int*>(at), reinterpret_cast<float*>(at) + room, reinterpret_cast<float*>(at) + 2 * room};
}

// A list's first entries, two a lane (four took more registers than a warp of the form by
// parts has, and what is spilled is waited for).
constexpr int kListAhead = 2;
template <typename T>
struct ListAhead {
  uint2 id[kListAhead];          // 64 bits, or the first 32 of them
  uint32_t value[kListAhead];    // 32 bits, or the first 16 of them
  Raw<T> z[kListAhead];
  float weight, grad_out;
};
// An id's column; -1: the list has ended, -2: not a column.
__device__ __forceinline__ int column_of(const RowLossParams& p, uint2 id) {
  const int64_t wide = p.ids32 ? static_cast<int>(id.x) : static_cast<int64_t>(static_cast<uint64_t>(id.y) << 32 | id.x);
  return wide < 0 ? -1 : wide < p.V ? static_cast<int>(wide) : -2;
}
__device__ __forceinline__ uint2 raw_id(const RowLossParams& p, int64_t i) {
  uint2 r = make_uint2(0, 0);
  if (p.ids32)
    r.x = __ldg(static_cast<const uint32_t*>(p.ids) + i);
  else
    r = __ldg(static_cast<const uint2*>(p.ids) + i);
  return r;
}
__device__ __forceinline__ uint32_t raw_value(const RowLossParams& p, int64_t i) {
  return p.value_dtype == FLCE_DTYPE_FP32 ? __ldg(static_cast<const uint32_t*>(p.values) + i)
                                          : __ldg(static_cast<const uint16_t*>(p.values) + i);
}
__device__ __forceinline__ float value_of(const RowLossParams& p, uint32_t raw) {
  return p.value_dtype == FLCE_DTYPE_FP32   ? __uint_as_float(raw)
         : p.value_dtype == FLCE_DTYPE_FP16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(raw)))
                                            : __uint_as_float(raw << 16);
}
template <typename T, int KIND>
__device__ __forceinline__ ListAhead<T> list_ahead(const RowLossParams& p, int64_t row) {
  ListAhead<T> a;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kListAhead; ++j) {
    const int k = j * 32 + lane;
    a.id[j] = make_uint2(0xFFFFFFFFu, 0xFFFFFFFFu);
    a.value[j] = 0;
    if (KIND == kDistill && row < p.N && k < p.K) {
      a.id[j] = raw_id(p, row * p.K + k);
      a.value[j] = raw_value(p, row * p.K + k);
    }
  }
  a.weight = a.grad_out = 1.f;
  if (row < p.N && p.row_weight != nullptr) a.weight = __ldg(p.row_weight + row);
  if (row < p.N && p.grad_out != nullptr) a.grad_out = __ldg(p.grad_out + row);
  return a;
}
template <typename T>
__device__ __forceinline__ void list_logits(const RowLossParams& p, int64_t row, ListAhead<T>& a) {
#pragma unroll
  for (int j = 0; j < kListAhead; ++j) {
    const int column = column_of(p, a.id[j]);
    if (column >= 0) a.z[j] = raw_logit<T>(p, row, column);
  }
}

// Puts a column into the table of a list, which has room for all; whether it was there.
__device__ __forceinline__ bool seen_before(int* table, int slots, int column) {
  for (unsigned s = (static_cast<unsigned>(column) * 2654435761u) >> 8;; ++s) {
    const int was = atomicCAS(table + (s & (slots - 1)), -1, column);
    if (was == -1) return false;
    if (was == column) return true;
  }
}

// Where a column is named twice: every entry gets its column's whole share, so that all that
// name it write the same.  `table` is free.
__device__ __forceinline__ void join_shares(const TeacherList& list, int entries, int* table) {
  float* total = reinterpret_cast<float*>(table);
  __syncwarp();
  for (int k = threadIdx.x & 31; k < entries; k += 32) {
    float q = 0.f;
    for (int j = 0; j < entries; ++j)
      if (list.column[j] == list.column[k]) q += list.q[j];
    total[k] = q;
  }
  __syncwarp();
  for (int k = threadIdx.x & 31; k < entries; k += 32) list.q[k] = total[k];
  __syncwarp();
}

// A list of up to 32 * kListAhead entries, without leaving the registers.
template <typename T, typename Wanted>
__device__ __forceinline__ RowInfo short_teacher_row(const RowLossParams& p, const ListAhead<T>& ahead,
                                                     const TeacherList& list, int* table, int* bits,
                                                     const Wanted& wanted) {
  const int lane = threadIdx.x & 31;
  RowInfo r = {};
  r.weight = ahead.weight;
  r.grad_out = ahead.grad_out;
  r.column = -1;
  const int slots = table_slots(p.K);
  for (int i = lane; i < slots; i += 32) table[i] = -1;
  __syncwarp();
  const int batches = (p.K + 31) / 32;
  float v[kListAhead], e[kListAhead], z[kListAhead];
  int column[kListAhead];
  float vmax = -INFINITY;
  bool ended = false;
#pragma unroll
  for (int j = 0; j < kListAhead; ++j) {
    v[j] = -INFINITY;
    if (j >= batches) break;
    column[j] = column_of(p, ahead.id[j]);
    z[j] = raw_float<T>(ahead.z[j]);
    const unsigned ends = __ballot_sync(0xffffffffu, column[j] == -1);
    const bool held = !ended && (ends == 0 || lane < __ffs(ends) - 1);
    if (held && column[j] == -2) *bits |= FLCE_STATUS_BIT_TARGET_RANGE;
    if (held && column[j] >= 0) v[j] = value_of(p, ahead.value[j]);
    ended = ended || ends != 0;
    vmax = fmaxf(vmax, v[j]);
  }
  vmax = warp_max_redux(vmax);
  const float shift = vmax > -INFINITY ? vmax : 0.f;
  float sum = 0.f, zmax = -INFINITY;
#pragma unroll
  for (int j = 0; j < kListAhead; ++j) {
    e[j] = 0.f;
    if (j >= batches) break;
    e[j] = ex2_approx((v[j] - shift) * p.c);  // 0: no share, the place is like any other
    sum += e[j];
    if (e[j] != 0.f) zmax = fmaxf(zmax, z[j]);
  }
  sum = warp_sum(sum);
  zmax = warp_max_redux(zmax);
  r.zt = zmax > -INFINITY ? zmax : 0.f;
  r.taught = sum != 0.f;  // (a list of -inf alone is no teacher)
  const float inv = 1.f / sum, ln_sum = logf(sum);
  float a = 0.f;
  bool twice = false;
  int kept = 0;
#pragma unroll
  for (int j = 0; j < kListAhead; ++j) {
    if (j >= batches) break;
    const bool held = e[j] != 0.f;
    const float q = e[j] * inv;
    if (held) {
      a += q * ((v[j] - shift) * p.inv_t - ln_sum - (z[j] - r.zt) * p.inv_t);
    }
    const bool here = held && wanted(column[j]);
    if (here) twice = seen_before(table, slots, column[j]) || twice;
    const unsigned all = __ballot_sync(0xffffffffu, here);
    if (here) {
      const int at = kept + __popc(all & ((1u << lane) - 1));
      list.column[at] = column[j], list.q[at] = q, list.z[at] = z[j];
    }
    kept += __popc(all);
  }
  r.a = warp_sum(a);
  r.entries = kept;
  if (__any_sync(0xffffffffu, twice)) join_shares(list, kept, table);
  __syncwarp();
  return r;
}

// Any list, through shared memory.
template <typename T, typename Wanted>
__device__ __forceinline__ RowInfo long_teacher_row(const RowLossParams& p, int64_t row, float weight, float grad_out,
                                                    const TeacherList& list, int* table, int* bits,
                                                    const Wanted& wanted) {
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 31;
  const int64_t base = row * p.K;
  RowInfo r = {};
  r.weight = weight;
  r.grad_out = grad_out;
  r.column = -1;
  // ids and values, and where the list ends
  int entries = p.K;
  for (int k0 = 0; k0 < p.K; k0 += 32 * kBatch) {
    uint2 id[kBatch];
    uint32_t value[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j * 32 + lane;
      if (k < p.K) id[j] = raw_id(p, base + k), value[j] = raw_value(p, base + k);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j * 32 + lane;
      if (k >= p.K) break;
      const int column = column_of(p, id[j]);
      list.column[k] = column;
      list.q[k] = column >= 0 ? value_of(p, value[j]) : -INFINITY;
      if (column == -1) entries = min(entries, k);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) entries = min(entries, __shfl_xor_sync(0xffffffffu, entries, o));
  __syncwarp();
  float vmax = -INFINITY;
  for (int k = lane; k < entries; k += 32) {
    if (list.column[k] < 0) *bits |= FLCE_STATUS_BIT_TARGET_RANGE;
    vmax = fmaxf(vmax, list.q[k]);
  }
  vmax = warp_max_redux(vmax);
  const float shift = vmax > -INFINITY ? vmax : 0.f;
  // sum e, and sum e ((v - shift) - (z - zt)) / T with zt the largest logit of a lane's entries
  // so far, and then of all lanes' (another one, which a mask has put far below the rest, would
  // take the digits of the sum); the wanted entries move to the front of the list, to places
  // that have been read
  float sum = 0.f, a = 0.f, zt = -FLT_MAX;
  int kept = 0;
  for (int k0 = 0; k0 < entries; k0 += 32 * kBatch) {
    int column[kBatch];
    float v[kBatch];
    Raw<T> raw[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j * 32 + lane;
      column[j] = k < entries ? list.column[k] : -1;
      v[j] = k < entries ? list.q[k] - shift : -INFINITY;
      if (column[j] >= 0) raw[j] = raw_logit<T>(p, row, column[j]);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (k0 + j * 32 >= entries) break;
      const float e = ex2_approx(v[j] * p.c);  // 0: no share, the place is like any other
      const bool held = column[j] >= 0 && e != 0.f;
      const float z = held ? raw_float<T>(raw[j]) : 0.f;
      if (held) {
        if (z > zt) {
          if (sum != 0.f) a += sum * ((z - zt) * p.inv_t);
          zt = z;
        }
        sum += e;
        a += e * ((v[j] - (z - zt)) * p.inv_t);
      }
      const bool here = held && wanted(column[j]);
      const unsigned all = __ballot_sync(0xffffffffu, here);
      if (here) {
        const int at = kept + __popc(all & ((1u << lane) - 1));
        list.column[at] = column[j], list.q[at] = e, list.z[at] = z;
      }
      kept += __popc(all);
    }
    __syncwarp();
  }
  r.zt = warp_max_redux(zt);
  if (sum != 0.f) a += sum * ((r.zt - zt) * p.inv_t);
  sum = warp_sum(sum);
  r.taught = sum != 0.f;  // (a list of -inf alone is no teacher)
  r.entries = r.taught ? kept : 0;
  const float inv = 1.f / sum;
  r.a = warp_sum(a) * inv - logf(sum);
  // a column that is named twice is twice among the wanted entries
  const int slots = table_slots(p.K);
  for (int i = lane; i < slots; i += 32) table[i] = -1;
  __syncwarp();
  bool twice = false;
  for (int k = lane; k < r.entries; k += 32) {
    list.q[k] *= inv;
    twice = seen_before(table, slots, list.column[k]) || twice;
  }
  if (__any_sync(0xffffffffu, twice)) join_shares(list, r.entries, table);
  __syncwarp();
  return r;
}

// A row's list, by one warp: returns the row's numbers and fills `list` with the entries
// whose columns are `wanted`, q of columns that occur twice added up.  `ahead`: the list's
// first entries, with their logits.  `table` has table_slots(K) words.
template <typename T, int KIND, typename Wanted>
__device__ __forceinline__ RowInfo teacher_row(const RowLossParams& p, int64_t row, const ListAhead<T>& ahead,
                                               const TeacherList& list, int* table, int* bits, const Wanted& wanted) {
  if constexpr (KIND == kDistill)
    return short_teacher_row<T>(p, ahead, list, table, bits, wanted);
  else
    return long_teacher_row<T>(p, row, ahead.weight, ahead.grad_out, list, table, bits, wanted);
}
template <typename T, int KIND>
__device__ __forceinline__ RowInfo whole_teacher_row(const RowLossParams& p, int64_t row, const TeacherList& list,
                                                     int* table, int* bits) {
  ListAhead<T> a = list_ahead<T, KIND>(p, row);
  if constexpr (KIND == kDistill) list_logits<T>(p, row, a);
  return teacher_row<T, KIND>(p, row, a, list, table, bits, [](int) { return true; });
}

// ---------------------------------------------------------------- a row's loss

struct RowResult {
  float loss, logp;
  float f;  // the gradient is f (p - ...); 0: the row's gradient is 0 whatever its logits
};

// What a + b loses as its fp32 sum is rounded (Knuth's two-sum), 0 where that is no number.
__device__ __forceinline__ float sum_error(float a, float b, float sum) {
  const float from_b = sum - a;
  const float e = (a - (sum - from_b)) + (b - from_b);
  return fabsf(sum) < INFINITY ? e : 0.f;
}

// (zt - m) / T - ln s as `high` plus `low`.  A log-probability of -12 is rounded by 5e-7 in fp32,
// and a policy's loss knows it by its difference to another one of that size, which takes these
// digits whole: with the rest apart that difference is as good as s is.  ln s goes by s's own
// exponent, whose multiple of ln 2 is split so that its larger part is exact.
struct LogP {
  float high, low;
};
__device__ __forceinline__ LogP split_logp(const RowLossParams& p, float zt, float m, float s) {
  constexpr float kLn2High = 2839.f / 4096.f;  // 12 bits: exact times an exponent
  constexpr float kLn2Low = 3.194618494528623e-5f;
  const int k = (__float_as_int(s) >> 23 & 255) - 127;
  const float f = s * __uint_as_float(static_cast<unsigned>(127 - k) << 23), exponent = static_cast<float>(k);
  const float d = zt - m, t = d * p.inv_t;
  const float rest = fabsf(t) < INFINITY ? fmaf(-t, p.temperature, d) + sum_error(zt, -m, d) : 0.f;
  LogP r;
  r.high = fmaf(-exponent, kLn2High, t);
  r.low = sum_error(t, -exponent * kLn2High, r.high) + rest * p.inv_t - fmaf(exponent, kLn2Low, logf(f));
  return r;
}

// `scale`: what multiplies all gradients (grad_scale, or that over the rows of a mean).
template <int KIND>
__device__ __forceinline__ RowResult row_result(const RowLossParams& p, const RowInfo& r, float m, float s,
                                                float scale) {
  RowResult out = {0.f, 0.f, 0.f};
  scale *= r.grad_out;
  if constexpr (has_list(KIND)) {
    if (!r.taught || r.weight == 0.f) return out;
    out.loss = p.temperature * p.temperature * r.weight * (r.a + ((m - r.zt) * p.inv_t + logf(s)));
    out.f = p.temperature * r.weight * scale;
  } else if constexpr (KIND == kStats) {
    if (r.column >= 0) out.logp = (r.zt - m) * p.inv_t - logf(s);
  } else {
    if (r.column < 0) return out;
    const LogP logp = split_logp(p, r.zt, m, s);
    out.logp = logp.high + logp.low;
    if (r.weight == 0.f) return out;
    const float a = r.advantage;
    // fresh samples have a ratio of 1, but a row of no number has none
    const float ratio = p.old_logp != nullptr ? expf((logp.high - r.old_logp) + logp.low)
                        : isnan(out.logp)     ? out.logp
                                              : 1.f;
    const bool over = a > 0.f && ratio > p.ratio_high, under = a < 0.f && ratio < p.ratio_low;
    // an advantage of 0 takes nothing of a ratio that fp32 holds as infinite (NaN stays)
    const float gain = a == 0.f && ratio > FLT_MAX ? 0.f : a * ratio;
    float loss = over ? -a * p.ratio_high : under ? -a * p.ratio_low : -gain;
    float slope = over || under ? 0.f : -gain;
    if (p.kl_weight != 0.f) {
      const float d = (r.ref_logp - logp.high) - logp.low, x = expm1f(d);
      loss += p.kl_weight * (x - d);
      slope -= p.kl_weight * x;
    }
    out.loss = loss * r.weight;
    out.f = -slope * r.weight * scale * p.inv_t;
  }
  return out;
}

// The gradient at a place that the row names.
__device__ __forceinline__ float target_grad(const RowResult& r) { return r.f * expm1f(r.logp); }
__device__ __forceinline__ float entry_grad(const RowLossParams& p, const TeacherList& list, int k, float f, float m,
                                            float inv_s) {
  return f * (ex2_approx((list.z[k] - m) * p.c) * inv_s - list.q[k]);
}

// ---------------------------------------------------------------- rows that take part, and the end

template <int KIND>
__device__ __forceinline__ bool takes_part(const RowLossParams& p, int64_t n) {
  if constexpr (has_list(KIND)) return load_id(p.ids, p.ids32, n * p.K) >= 0;
  const int64_t t = __ldg(p.target + n);
  return t != p.ignore_index && t >= 0 && t < p.V;
}

// Partial counts of rows n, n + step, ...: by one thread.
template <int KIND>
__device__ __forceinline__ int count_rows(const RowLossParams& p, int64_t n, int64_t step) {
  int count = 0;
#pragma unroll 4
  for (; n < p.N; n += step) count += takes_part<KIND>(p, n);
  return count;
}

template <int KIND>
__global__ void __launch_bounds__(256) row_count_kernel(const RowLossParams p, int* counts) {
  __shared__ int total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  const int mine = count_rows<KIND>(p, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, kCountCtas * 256);
  if (mine != 0) atomicAdd(&total, mine);
  __syncthreads();
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// The rows of a mean, in every lane of a warp, from row_count_kernel's counts.
__device__ __forceinline__ int counted_rows(const int* counts) {
  int n = 0;
  for (int i = threadIdx.x & 31; i < kCountCtas; i += 32) n += __ldcg(counts + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// By all threads of every CTA of a launch, at its end: adds up the CTAs' losses (of thread
// 0) in the order of the CTAs, and their status bits, in the CTA that arrives last.  One
// warp adds: an SM has two fp64 operations a cycle.
__device__ __forceinline__ void finish_rows(const RowLossParams& p, double loss, int bits, int rows) {
  __shared__ int last;
  constexpr unsigned kStaged = 256;
  __shared__ double staged[kStaged];
  __shared__ int all_bits;
  if (threadIdx.x == 0) {
    all_bits = 0;
    if (p.loss != nullptr) p.partial[blockIdx.x] = loss;
    p.flags[blockIdx.x] = bits;
    last = arrives_last(p.arrivals, p.tag, gridDim.x);
  }
  __syncthreads();
  if (!last) return;
  int seen = 0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += blockDim.x) seen |= __ldcg(p.flags + i);
  double total = 0;
  for (unsigned base = 0; base < gridDim.x && p.loss != nullptr; base += kStaged) {
    const unsigned here = gridDim.x - base < kStaged ? gridDim.x - base : kStaged;
    for (unsigned i = threadIdx.x; i < here; i += blockDim.x) staged[i] = __ldcg(p.partial + base + i);
    __syncthreads();
    if (threadIdx.x < 32)
      for (unsigned i = threadIdx.x; i < here; i += 32) total += staged[i];
    __syncthreads();
  }
  if (seen != 0) atomicOr(&all_bits, seen);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  if (p.loss != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (threadIdx.x != 0) return;
  if (p.loss != nullptr)
    *p.loss = p.reduction != FLCE_REDUCTION_MEAN ? static_cast<float>(total)
              : rows > 0                         ? static_cast<float>(total / rows)
                                                 : __int_as_float(0x7fc00000);
  if (p.own_status)
    *p.status = all_bits;
  else if (all_bits != 0)
    atomicOr(p.status, all_bits);
}

// What a row's result leaves beside its gradient: by one thread.
template <int KIND>
__device__ __forceinline__ void store_result(const RowLossParams& p, int64_t row, const RowResult& r, float m,
                                             float s, double* loss) {
  if constexpr (KIND == kStats) {
    p.stats[row] = make_float2(m, 1.f / s);
    p.factor[row] = 0.f;
  } else {
    *loss += r.loss;
    if (p.loss_rows != nullptr) p.loss_rows[row] = r.loss;
  }
  if (p.logp != nullptr) p.logp[row] = r.logp;
}

// ---------------------------------------------------------------- rows of any length

// One CTA a row, which reads it twice: for rows that the form by parts does not hold (more
// than 512 KB).  Two readings and a write bound it: fp32 [1000, 256000] 539 us, of which L2
// gives some of the second reading (301 would be one reading at the copy rate).
constexpr int kLongThreads = 512;
constexpr int kLongVecs = 4;
constexpr int kLongBatch = 64;  // steps whose sums are added up before they join the rest, for short chains

template <typename T, int KIND>
__global__ void __launch_bounds__(kLongThreads) row_loss_long_kernel(const RowLossParams p) {
  extern __shared__ __align__(16) uint8_t list_memory[];
  constexpr int kWarps = kLongThreads / 32, kE = kVecElems<T>;
  __shared__ RowInfo info;
  __shared__ float2 parts[kWarps];
  __shared__ int count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TeacherList list = list_at(list_memory, p.K);
  if (tid == 0) {
    count = 0;
    if (blockIdx.x == 0) expect_arrivals(p.arrivals, p.tag);
  }
  __syncthreads();
  int rows = 1, bits = 0;
  grid_dependency_wait();
  if (p.reduction == FLCE_REDUCTION_MEAN) {
    if (p.counts != nullptr) {
      rows = counted_rows(p.counts);
    } else {
      const int mine = count_rows<KIND>(p, tid, kLongThreads);
      if (mine != 0) atomicAdd(&count, mine);
      __syncthreads();
      rows = count;
    }
  }
  const float scale = p.reduction == FLCE_REDUCTION_MEAN ? p.grad_scale / static_cast<float>(rows) : p.grad_scale;
  const Pair c = pair(p.c);
  double loss = 0;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const RowSplit split = split_row(x, p.V);
    const uint4* vecs = reinterpret_cast<const uint4*>(x + split.head);
    const T* tail = x + split.head + static_cast<int64_t>(split.vecs) * kE;
    float m = -INFINITY, s = 0.f;
    if (warp == 0) {
      RowInfo r;
      if constexpr (has_list(KIND))
        r = whole_teacher_row<T, KIND>(p, row, list, reinterpret_cast<int*>(list_memory + list_bytes(p.K)), &bits);
      else
        r = policy_row<T>(p, row, &bits);
      if (lane == 0) info = r;
    }
    if (tid < split.head) m = to_float(x[tid]), s = 1.f;
    if (tid >= 32 && tid < 32 + split.tail) m = to_float(tail[tid - 32]), s = 1.f;
    if (s == 1.f && !(m > -INFINITY)) s = m == m ? 0.f : m;  // -inf adds nothing, NaN stays
    float whole = 0.f;  // of the batches of kLongBatch steps that are done, by the same m
    int step = 0;
    for (int64_t at = tid; at < split.vecs; at += kLongThreads * kLongVecs) {
      uint4 v[kLongVecs];
#pragma unroll
      for (int i = 0; i < kLongVecs; ++i) {
        const int64_t k = at + i * kLongThreads;
        v[i] = k < split.vecs ? vecs[k] : empty_vec<T>();
      }
      const float top = fmaxf(m, vecs_max<T, kLongVecs>(v));
      const float shift = top > -INFINITY ? top : 0.f;
      Pair sum = pair(0.f);
#pragma unroll
      for (int i = 0; i < kLongVecs; ++i) vec_add_exp<T>(v[i], pair(-shift), c, sum);
      const float2 both = unpair(sum);
      const float less = m > -INFINITY ? ex2_approx((m - shift) * p.c) : 1.f;
      s = s * less + (both.x + both.y);
      whole *= less;
      m = top;
      if (++step % kLongBatch == 0) whole += s, s = 0.f;
    }
    const float2 mine = combine_parts(m, s + whole, p.c);
    if (lane == 0) parts[warp] = mine;
    __syncthreads();
    const float2 part = lane < kWarps ? parts[lane] : make_float2(-INFINITY, 0.f);
    const float2 all = combine_parts(part.x, part.y, p.c);
    const RowInfo r = info;
    const RowResult result = row_result<KIND>(p, r, all.x, all.y, scale);
    if (tid == 0) store_result<KIND>(p, row, result, all.x, all.y, &loss);
    if (KIND != kStats && p.grad != nullptr) {
      T* g = static_cast<T*>(p.grad) + row * p.ld_grad;
      const float inv_s = 1.f / all.y, f = result.f * inv_s;
      const Pair minus_m = pair(-all.x), factor = pair(f);
      const bool zero = result.f == 0.f, vector = same_phase(x, g);
      if (tid < split.head) g[tid] = from_float<T>(zero ? 0.f : f * ex2_approx((to_float(x[tid]) - all.x) * p.c));
      if (tid >= 32 && tid < 32 + split.tail) {
        const int64_t at = p.V - split.tail + tid - 32;
        g[at] = from_float<T>(zero ? 0.f : f * ex2_approx((to_float(x[at]) - all.x) * p.c));
      }
#pragma unroll 4
      for (int64_t at = tid; at < split.vecs; at += kLongThreads) {
        const uint4 v = zero ? make_uint4(0, 0, 0, 0) : vec_grad<T>(__ldcs(vecs + at), minus_m, c, factor);
        store_vec<T>(g + split.head + at * kE, v, vector);
      }
      __syncthreads();  // the places that the row names are written after the rest
      if (!zero) {
        if constexpr (has_list(KIND)) {
          for (int k = tid; k < r.entries; k += kLongThreads)
            g[list.column[k]] = from_float<T>(entry_grad(p, list, k, result.f, all.x, inv_s));
        } else if (tid == 0) {
          g[r.column] = from_float<T>(target_grad(result));
        }
      }
    }
    __syncthreads();  // info, list and parts are the next row's
  }
  if (warp == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
  }
  finish_rows(p, loss, bits, rows);
}

template <typename T, int KIND>
cudaError_t launch_long(const RowLossParams& p, cudaStream_t s) {
  const size_t smem = has_list(KIND) ? list_bytes(p.K) + table_slots(p.K) * 4 : 0;
  const int64_t most = 4 * device_sm_count();
  const unsigned grid = static_cast<unsigned>(p.N < 1 ? 1 : p.N < most ? p.N : most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kLongThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.counts != nullptr ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, row_loss_long_kernel<T, KIND>, p);
}

// ---------------------------------------------------------------- short rows

// A warp a row, which it holds in registers: rows of up to 512 vectors.  Bound by what a row
// costs beside its elements: bf16 [65536, 2048] 115 us against 79 at the copy rate, [32768,
// 4096] 120 against 79.  CTAs of eight warps, but of four where a thread's 16 vectors take 168
// registers, of which an SM has room for 12 warps (with eight: 152 us; four for eight vectors
// made fp32 [65536, 1000] 92 -> 110).
constexpr int row_warps(int vecs) { return vecs > 8 ? 4 : 8; }

template <typename T, int KIND, int VPT>
__global__ void __launch_bounds__(32 * row_warps(VPT)) row_loss_warps_kernel(const RowLossParams p) {
  extern __shared__ __align__(16) uint8_t list_memory[];
  constexpr int kE = kVecElems<T>;
  __shared__ double losses[row_warps(VPT)];
  __shared__ int count, all_bits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const size_t each = has_list(KIND) ? list_bytes(p.K) + table_slots(p.K) * 4 : 0;
  const TeacherList list = list_at(list_memory + warp * each, p.K);
  int* const table = reinterpret_cast<int*>(list_memory + warp * each + list_bytes(p.K));
  if (tid == 0) {
    count = all_bits = 0;
    if (blockIdx.x == 0) expect_arrivals(p.arrivals, p.tag);
  }
  int rows = 1, bits = 0;
  const bool mean = p.reduction == FLCE_REDUCTION_MEAN && KIND != kStats;
  const bool self = mean && p.counts == nullptr;
  if (self) {
    __syncthreads();
    int n = count_rows<KIND>(p, tid, blockDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0 && n != 0) atomicAdd(&count, n);
  }
  __syncthreads();
  if (self) rows = count;
  if (mean && !self) {
    grid_dependency_wait();
    rows = counted_rows(p.counts);
  }
  const float scale = mean ? p.grad_scale / static_cast<float>(rows) : p.grad_scale;
  const Pair c = pair(p.c);
  double loss = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * warps + warp; row < p.N;
       row += static_cast<int64_t>(gridDim.x) * warps) {
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const RowSplit split = split_row(x, p.V);
    const int n = static_cast<int>(split.vecs);
    const uint4* from = reinterpret_cast<const uint4*>(x + split.head);
    uint4 v[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) v[k] = k * 32 + lane < n ? from[k * 32 + lane] : empty_vec<T>();
    int extra = -1;  // an element before or after the vectors
    if (lane < split.head) extra = lane;
    if (lane >= 8 && lane < 8 + split.tail) extra = static_cast<int>(p.V) - split.tail + lane - 8;
    const float z = extra >= 0 ? to_float(x[extra]) : -INFINITY;
    RowInfo r;
    if constexpr (has_list(KIND))
      r = whole_teacher_row<T, KIND>(p, row, list, table, &bits);
    else
      r = policy_row<T>(p, row, &bits);
    const float m = warp_max_redux(fmaxf(vecs_max<T, VPT>(v), z));
    const Pair minus_m = pair(m > -INFINITY ? -m : 0.f);
    Pair sum = pair(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) vec_add_exp<T>(v[k], minus_m, c, sum);
    float2 both = unpair(sum);
    if (extra >= 0) both.x += ex2_approx((z + unpair(minus_m).x) * p.c);
    const float s = warp_sum(both.x + both.y);
    const RowResult result = row_result<KIND>(p, r, m, s, scale);
    if (lane == 0) store_result<KIND>(p, row, result, m, s, &loss);
    if (KIND == kStats || p.grad == nullptr) continue;
    T* g = static_cast<T*>(p.grad) + row * p.ld_grad;
    const bool zero = result.f == 0.f, vector = same_phase(x, g);
    const float inv_s = 1.f / s, f = result.f * inv_s;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint4 out = zero ? make_uint4(0, 0, 0, 0) : vec_grad<T>(v[k], pair(-m), c, pair(f));
      if (k * 32 + lane < n) store_vec<T>(g + split.head + (k * 32 + lane) * kE, out, vector);
    }
    if (extra >= 0) g[extra] = from_float<T>(zero ? 0.f : f * ex2_approx((z - m) * p.c));
    __syncwarp();  // the places that the row names are written after the rest
    if (zero) continue;
    if constexpr (has_list(KIND)) {
      for (int k = lane; k < r.entries; k += 32)
        g[list.column[k]] = from_float<T>(entry_grad(p, list, k, result.f, m, inv_s));
      __syncwarp();  // the list is the next row's
    } else if (lane == 0) {
      g[r.column] = from_float<T>(target_grad(result));
    }
  }
  if (lane == 0) losses[warp] = loss;
  if (bits != 0) atomicOr(&all_bits, bits);
  __syncthreads();
  double total = 0;
  if (tid == 0 && p.loss != nullptr)
    for (int w = 0; w < warps; ++w) total += losses[w];
  finish_rows(p, total, all_bits, rows);
}

template <typename T, int KIND, int VPT>
cudaError_t launch_warps(const RowLossParams& p, cudaStream_t s) {
  const size_t each = has_list(KIND) ? list_bytes(p.K) + table_slots(p.K) * 4 : 0;
  int warps = row_warps(VPT);  // fewer where the lists are long, or the rows few
  while (warps > 1 && (warps * each > 40 * 1024 || div_up(p.N, warps) < device_sm_count())) warps /= 2;
  const int64_t ctas = div_up(p.N, warps), most = 8 * device_sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = warps * each;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.counts != nullptr ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, row_loss_warps_kernel<T, KIND, VPT>, p);
}

// ---------------------------------------------------------------- rows by parts

// A cluster of CTAs a row, each with one part of it in registers, so that a row is read
// once.  Clusters take rows one after another; CTAs of several clusters share an SM, and
// one computes while another waits.  The roles of a CTA's warps:
//
//   leader    brings the CTA's parts of the next rows into shared memory by bulk copies, and
//             reads what the rows have beside their logits
//   others    copy a part into registers, which frees its place, find its maximum and sum,
//             and hand both to every CTA of the row (one 8-byte store a warp and CTA, counted
//             by the receiver's barrier); later they write the gradient from the registers
//   closer    adds up the row's partial sums, and works out its loss and factors once for all
//             (done by every warp it took half of the kernel's instructions); it also has the
//             elements before the row's first vector and after its last
//
// Exponents here are x = z c - r with c = log2(e) / T and r = m c rounded: one rounding, of x
// itself, as z c - r is one operation, so that a common level takes no digits.  At z = m this
// leaves x = m c - r, up to half a unit in the last place of r, for the sums' last step to take
// out: at most 64 below |m c| = 2^31, so that sums stay between 2^-64 and V 2^64.  (Shares below
// 2^-62 of the largest may vanish where the row's maximum lies there; at 2^20 those below 2^-125.)
// From 2^31 on 2^x could overflow, and any two different fp32 logits are 2^31 2^-24 = 2^7 apart in
// x, which leaves no share: the warp replaces its z by z - m, and r by 0, and warps with other
// maxima have no share in the row.  (So from 2^20 on, and what joins warps exact at any distance:
// bf16 [4096, 128256] without gradients 213 -> 222 us, with masks of -1e9 330 -> 351.)
//
// Bound by memory where rows are many and long: bf16 [4096, 128256] 328 us for the policy loss
// and as much for a teacher's 64 entries, 94 % of the copy rate; fp32 [1000, 50257] 72 us, 82 %,
// as its last rows leave half of the SMs idle.  Rows of 8 to 32 KB cost their exchange of sums
// and the closer's arithmetic, 60 to 80 % of the copy rate.  Few rows cost what one does: bf16
// [1, 128256] 10.4 us, [256, 1024] (by warps) 7.9 on the GPU.
constexpr int kPartSlots = 4;
constexpr float kFarExponent = 2147483648.f;  // 2^31

struct PartShape {
  int cluster;    // CTAs of a row
  int seg_vecs;   // vectors of a part
  int slots;      // parts in shared memory
  int slot_bytes;
};

// What the closer leaves for the CTA's other warps.
struct PartResult {
  float m, r;       // the row's maximum; its exponent
  float factor;     // gradient of an element: factor 2^x
  float f, inv_s;   // f and 1 / S, S by the maximum itself
  float named;      // policy: the gradient at the target
  int column;       // policy: the target's, or -1
  int entries;
};

__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "l"(reinterpret_cast<uint64_t>(from)), "r"(bytes), "r"(bar)
               : "memory");
}
// Two floats to another CTA's shared memory, counted on its barrier.
__device__ __forceinline__ void push_pair(uint32_t to, float a, float b, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(a),
               "f"(b), "r"(bar)
               : "memory");
}

__device__ __forceinline__ bool far_exponent(float m, float c) { return !(fabsf(m * c) < kFarExponent); }

// 2^(z c - r) of a vector's elements.
template <typename T>
__device__ __forceinline__ void vec_exp2(const uint4& v, Pair c, Pair minus_r, Pair (&e)[kVecElems<T> / 2]) {
  vec_pairs<T>(v, e);
#pragma unroll
  for (int k = 0; k < kVecElems<T> / 2; ++k) {
    const float2 x = unpair(fma_pair(e[k], c, minus_r));
    e[k] = pair(ex2_approx(x.x), ex2_approx(x.y));
  }
}

// Elements z of a vector become z - m.
template <typename T>
__device__ __forceinline__ void vec_subtract(uint4& v, float m) {
  Pair e[kVecElems<T> / 2];
  vec_pairs<T>(v, e);
#pragma unroll
  for (int k = 0; k < kVecElems<T> / 2; ++k) e[k] = e[k] + pair(-m);
  v = pack_pairs<T>(e);
}

// A row of whole vectors.
template <typename T>
__device__ __forceinline__ RowSplit whole_row(int64_t V) {
  return {0, 0, static_cast<int>(static_cast<unsigned>(V) / kVecElems<T>)};
}

// THREADS: of the warps that compute; VPT: vectors a thread holds; WHOLE: all rows are whole
// vectors, in both matrices (what a row's place costs its threads was a fifth of their time).
template <typename T, int KIND, int THREADS, int VPT, int CTAS_PER_SM, bool WHOLE>
__global__ void __launch_bounds__(THREADS + 64, CTAS_PER_SM)
    row_loss_parts_kernel(const RowLossParams p, const PartShape shape) {
  constexpr int kE = kVecElems<T>, kWarps = THREADS / 32, kSums = kWarps + 1;
  constexpr int kKept = KIND == kStats ? 4 : 2;  // rows whose numbers a CTA keeps
  extern __shared__ __align__(128) uint8_t part_memory[];
  __shared__ uint64_t full[kPartSlots], empty[kPartSlots], told[kKept], summed[kKept], closed[kKept];
  __shared__ RowInfo infos[kKept];
  __shared__ PartResult results[kKept];
  __shared__ float2 parts[kKept][8 * kSums];  // (maximum, sum) of every warp of the row's CTAs; the closers' are empty
  __shared__ int aborted, count, all_bits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = shape.cluster;
  const int rank = static_cast<int>(cluster_cta_rank());
  const int first_row = static_cast<int>(blockIdx.x) / cluster, row_step = static_cast<int>(gridDim.x) / cluster;
  const int mine = p.N > first_row ? static_cast<int>((p.N - 1 - first_row) / row_step) + 1 : 0;
  uint8_t* const lists = part_memory + static_cast<size_t>(shape.slots) * shape.slot_bytes;
  if (tid == 0) {
    for (int i = 0; i < kPartSlots; ++i) {
      mbar_init(smem_addr(&full[i]), 1);
      mbar_init(smem_addr(&empty[i]), kWarps + (has_list(KIND) ? 1 : 0));
    }
    for (int i = 0; i < kKept; ++i) {
      mbar_init(smem_addr(&told[i]), 1);
      mbar_init(smem_addr(&summed[i]), 1);
      mbar_init(smem_addr(&closed[i]), 1);
    }
    aborted = count = all_bits = 0;
    fence_barrier_init();
    if (blockIdx.x == 0) expect_arrivals(p.arrivals, p.tag);
  }
  cluster_sync_all();  // (also the CTA's own barrier)
  // A wait that runs out leaves a status bit.  The warp that waited goes on through its rows, but no longer copies,
  // writes, or arrives at a barrier that others arrive at too (its last phase may not be over); the others' waits end
  // by the flag or run out, in the row's other CTAs as well.
  const WaitCtl ctl{&aborted, nullptr, p.timeout_ns};
  const auto row_of = [&](int i) { return static_cast<int64_t>(first_row) + static_cast<int64_t>(i) * row_step; };
  const auto logits_of = [&](int64_t row) { return static_cast<const T*>(p.logits) + row * p.ld; };
  const auto split_of = [&](const T* x) { return WHOLE ? whole_row<T>(p.V) : split_row(x, p.V); };
  const int first_vec = rank * shape.seg_vecs;
  const auto part_vecs = [&](const RowSplit& split) {
    const int left = split.vecs - first_vec;
    return left < 0 ? 0 : left < shape.seg_vecs ? left : shape.seg_vecs;
  };

  if (warp == kWarps) {
    // ------------------------------------------------ the leader
    int bits = 0, issued = 0, to_slot = 0;
    const auto issue = [&]() {  // the next row's part, by one lane
      const T* x = logits_of(row_of(issued));
      const RowSplit split = split_of(x);
      const uint32_t bytes = static_cast<uint32_t>(part_vecs(split)) * 16u;
      const uint32_t bar = smem_addr(&full[to_slot]);
      mbar_arrive_expect_tx(bar, bytes);
      if (bytes > 0)
        bulk_copy(smem_addr(part_memory) + to_slot * shape.slot_bytes,
                  reinterpret_cast<const uint4*>(x + split.head) + first_vec, bytes, bar);
      ++issued;
      if (++to_slot == shape.slots) to_slot = 0;
    };
    if (lane == 0)
      while (issued < shape.slots && issued < mine) issue();
    int slot = 0, use = 0;  // i % slots, i / slots
    const auto read_ahead = [&](int64_t row) {
      if constexpr (has_list(KIND))
        return list_ahead<T, KIND>(p, row);
      else
        return policy_ahead<T>(p, row);
    };
    const auto read_logits = [&](int64_t row, auto& a) {
      if constexpr (KIND == kDistill)
        list_logits<T>(p, row, a);
      else if constexpr (!has_list(KIND))
        policy_logit<T>(p, row, a);
    };
    auto ahead = read_ahead(row_of(0)), next = read_ahead(row_of(1));
    read_logits(row_of(0), ahead);
    for (int i = 0; i < mine; ++i) {
      // all warps have read row i - 1's part, so they have waited for row i - 2 to be closed (row i - 3 for kStats):
      // infos of row i - 4 and the list of row i - 2 are no longer used
      const int64_t row = row_of(i);
      RowInfo r;
      if constexpr (has_list(KIND)) {
        const size_t at = static_cast<size_t>(i & 1) * list_bytes(p.K);
        const RowSplit split = split_of(logits_of(row));
        const int n = part_vecs(split);
        r = teacher_row<T, KIND>(p, row, ahead, list_at(lists + at, p.K),
                           reinterpret_cast<int*>(lists + 2 * list_bytes(p.K)), &bits, [&](int column) {
                             const int inside = column - split.head, vec = inside / kE;
                             return inside < 0          ? rank == 0
                                    : vec >= split.vecs ? rank == cluster - 1
                                                        : vec >= first_vec && vec < first_vec + n;
                           });
      } else {
        r = policy_info<T>(p, ahead, &bits);
      }
      if (lane == 0) {
        infos[i % kKept] = r;
        mbar_arrive(smem_addr(&told[i % kKept]));
      }
      ahead = next;
      read_logits(row_of(i + 1), ahead);
      next = read_ahead(row_of(i + 2));
      if (lane == 0) {
        const bool read = mbar_wait_sleep(smem_addr(&empty[slot]), use & 1, ctl);
        if (read && !*ctl.abort_flag && issued < mine) issue();
      }
      if (++slot == shape.slots) slot = 0, ++use;
      __syncwarp();
    }
    if (lane == 0 && *ctl.abort_flag)  // copies under way have to land before this CTA ends
      for (int i = issued > shape.slots ? issued - shape.slots : 0; i < issued; ++i)
        mbar_wait_drain(smem_addr(&full[i % shape.slots]), (i / shape.slots) & 1, p.timeout_ns);
    if (bits != 0) atomicOr(&all_bits, bits);
  }

  double loss = 0;
  int rows = 1;
  if (warp == kWarps + 1) {
    // ------------------------------------------------ the closer
    if (p.reduction == FLCE_REDUCTION_MEAN && KIND != kStats) {
      if (p.counts != nullptr) {
        grid_dependency_wait();
        rows = counted_rows(p.counts);
      } else {
        asm volatile("barrier.sync 2, %0;" ::"n"(THREADS + 32) : "memory");  // the others have counted
        rows = count;
      }
    }
    const float scale = p.reduction == FLCE_REDUCTION_MEAN ? p.grad_scale / static_cast<float>(rows) : p.grad_scale;
    // its element of a row, if the CTA has one end of the row: read a row ahead
    const auto edge_of = [&](int i, int* at) -> float {
      *at = -1;
      if (WHOLE || i >= mine) return -INFINITY;
      const T* x = logits_of(row_of(i));
      const RowSplit split = split_of(x);
      if (rank == 0 && lane < split.head) *at = lane;
      if (rank == cluster - 1 && lane >= 8 && lane < 8 + split.tail) *at = static_cast<int>(p.V) - split.tail + lane - 8;
      return *at >= 0 ? to_float(x[*at]) : -INFINITY;
    };
    int edge, next_edge, slot = 0;
    float z, next_z = edge_of(0, &next_edge);
    bool alive = true;
    for (int i = 0; i < mine; ++i) {
      if (has_list(KIND) && lane == 0 && alive) mbar_arrive(smem_addr(&empty[slot]));  // done with row i - 1's list
      if (++slot == shape.slots) slot = 0;
      z = next_z, edge = next_edge;
      next_z = edge_of(i + 1, &next_edge);
      const int b = i % kKept, phase = (i / kKept) & 1;
      const uint32_t sum_bar = smem_addr(&summed[b]);
      if (lane == 0 && alive) mbar_arrive_expect_tx(sum_bar, static_cast<uint32_t>(cluster) * kSums * 8u);
      // no CTA may write a row (its logits may be in the same place) before all have read what they need of it:
      // this one's word for it is its closer's share in the sums
      alive = __all_sync(0xffffffffu, mbar_wait(smem_addr(&told[b]), phase, ctl)) && alive;
      float edge_m = -INFINITY, edge_s = 0.f;
      if constexpr (!WHOLE) {
        edge_m = warp_max_redux(z);
        // the same exponents as a part's (vec_exp2)
        const float taken = !(edge_m > -INFINITY) ? 0.f : __fmul_rn(edge_m, p.c);
        if (edge >= 0) edge_s = edge_m > -INFINITY && far_exponent(edge_m, p.c) ? ex2_approx((z - edge_m) * p.c)
                                                                               : ex2_approx(fmaf(z, p.c, -taken));
        edge_s = warp_sum(edge_s);
      }
      if (alive && lane < cluster)
        push_pair(map_to_cta(smem_addr(&parts[b][rank * kSums + kWarps]), lane), edge_m, edge_s,
                  map_to_cta(sum_bar, lane));
      const RowInfo info = infos[b];
      alive = __all_sync(0xffffffffu, mbar_wait_cluster(sum_bar, phase, ctl)) && alive;
      if (!alive) continue;
      float top = -INFINITY;
      for (int k = lane; k < cluster * kSums; k += 32) top = fmaxf(top, parts[b][k].x);
      const float m = warp_max_redux(top);
      const bool far = far_exponent(m, p.c);
      const float r = far ? 0.f : __fmul_rn(m, p.c);
      float sum = 0.f;
      for (int k = lane; k < cluster * kSums; k += 32) {
        const float2 q = parts[b][k];
        // a warp's sum goes by its own rounded exponent; warps that have found nothing have 0, or NaN
        const float scaled = q.y * ex2_approx(far ? (q.x == m ? 0.f : -INFINITY) : __fmul_rn(q.x, p.c) - r);
        sum += q.x > -INFINITY ? scaled : q.y;
      }
      sum = warp_sum(sum);                                        // of 2^(z c - r)
      const float s = far ? sum : sum * ex2_approx(fmaf(-m, p.c, r));  // of 2^((z - m) c)
      const RowResult result = row_result<KIND>(p, info, m, s, scale);
      if (lane == 0) {
        if (rank == 0) store_result<KIND>(p, row_of(i), result, m, s, &loss);
        PartResult out;
        out.m = m, out.r = r, out.f = result.f, out.inv_s = 1.f / s, out.factor = result.f / sum;
        out.named = KIND == kPolicy ? target_grad(result) : 0.f;
        out.column = info.column, out.entries = info.entries;
        results[b] = out;
        mbar_arrive(smem_addr(&closed[b]));
      }
      __syncwarp();
      if (!WHOLE && KIND != kStats && p.grad != nullptr) {
        T* g = static_cast<T*>(p.grad) + row_of(i) * p.ld_grad;
        const bool zero = result.f == 0.f;
        if (edge >= 0) {
          float out = zero ? 0.f : result.f * (1.f / s) * ex2_approx((z - m) * p.c);
          if (KIND == kPolicy && !zero && edge == info.column) out = target_grad(result);
          g[edge] = from_float<T>(out);
        }
        if constexpr (has_list(KIND)) {
          __syncwarp();  // the places that the row names are written after the rest
          if (!zero) {
            const RowSplit split = split_of(logits_of(row_of(i)));
            const TeacherList list = list_at(lists + static_cast<size_t>(i & 1) * list_bytes(p.K), p.K);
            for (int k = lane; k < info.entries; k += 32) {
              const int column = list.column[k];
              if (column < split.head || column >= static_cast<int>(p.V) - split.tail)
                g[column] = from_float<T>(entry_grad(p, list, k, result.f, m, 1.f / s));
            }
          }
          __syncwarp();
        }
      }
    }
  }

  if (warp < kWarps) {
    // ------------------------------------------------ the others
    if (p.reduction == FLCE_REDUCTION_MEAN && KIND != kStats && p.counts == nullptr) {
      int n = count_rows<KIND>(p, tid, THREADS);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == 0 && n != 0) atomicAdd(&count, n);
      asm volatile("barrier.sync 2, %0;" ::"n"(THREADS + 32) : "memory");
    }
    const Pair c = pair(p.c);
    int slot = 0, use = 0;
    const T* x = logits_of(first_row);
    T* g = static_cast<T*>(p.grad) + first_row * p.ld_grad;
    const int64_t x_step = row_step * p.ld, g_step = row_step * p.ld_grad;
    RowSplit split = split_of(x);
    int n = part_vecs(split);
    bool alive = true;
    for (int i = 0; i < mine; ++i, x += x_step, g += g_step) {
      if constexpr (!WHOLE) {
        split = split_of(x);
        n = part_vecs(split);
      }
      const int b = i % kKept, phase = (i / kKept) & 1;
      alive = mbar_wait_sleep(smem_addr(&full[slot]), use & 1, ctl) && alive;
      const uint4* from = reinterpret_cast<const uint4*>(part_memory + slot * shape.slot_bytes);
      uint4 v[VPT];
#pragma unroll
      for (int k = 0; k < VPT; ++k) v[k] = k * THREADS + tid < n ? from[k * THREADS + tid] : empty_vec<T>();
      __syncwarp();
      if (lane == 0 && alive) mbar_arrive(smem_addr(&empty[slot]));
      if (++slot == shape.slots) slot = 0, ++use;
      const float m = warp_max_redux(vecs_max<T, VPT>(v));
      const bool far = m > -INFINITY && far_exponent(m, p.c);
      if (far) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) vec_subtract<T>(v[k], m);
      }
      float r = far || !(m > -INFINITY) ? 0.f : __fmul_rn(m, p.c);
      Pair sum = pair(0.f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        Pair e[kE / 2];
        vec_exp2<T>(v[k], c, pair(-r), e);
#pragma unroll
        for (int q = 0; q < kE / 2; ++q) sum = sum + e[q];
      }
      const float2 both = unpair(sum);
      const float s = warp_sum(both.x + both.y);
      if (alive && lane < cluster)
        push_pair(map_to_cta(smem_addr(&parts[b][rank * kSums + warp]), lane), m, s,
                  map_to_cta(smem_addr(&summed[b]), lane));
      if constexpr (KIND == kStats) {
        // a row is closed while the next one is read.  What a row's sums overwrite, the row's four before, is no
        // longer wanted: row i - 1 closed here means that every CTA has closed row i - 2
        if (i > 0) alive = mbar_wait_sleep(smem_addr(&closed[(i - 1) % kKept]), ((i - 1) / kKept) & 1, ctl) && alive;
        continue;
      }
      alive = mbar_wait_sleep(smem_addr(&closed[b]), phase, ctl) && alive;
      if (p.grad == nullptr || !alive) continue;
      const PartResult result = results[b];
      const bool zero = result.f == 0.f;
      // a warp that has taken its own maximum off: the row's, or far below it
      r = !far ? result.r : m == result.m ? 0.f : INFINITY;
      if (!far && far_exponent(result.m, p.c)) r = result.m > 0.f ? INFINITY : 0.f;
      const Pair minus_r = pair(-r), factor = pair(result.factor);
      T* to = g + split.head + (static_cast<int64_t>(first_vec) + tid) * kE;
      // the 16-bit elements are widened again: kept from the sum, they would not fit in the registers
#pragma unroll
      for (int k = 0; k < VPT; ++k) asm volatile("" : "+r"(v[k].x), "+r"(v[k].y), "+r"(v[k].z), "+r"(v[k].w));
      const auto gradient = [&](const uint4& vec) {
        if (zero) return make_uint4(0, 0, 0, 0);
        Pair e[kE / 2];
        vec_exp2<T>(vec, c, minus_r, e);
#pragma unroll
        for (int q = 0; q < kE / 2; ++q) e[q] = e[q] * factor;
        return pack_pairs<T>(e);
      };
      if (WHOLE || same_phase(x, g)) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const uint4 out = gradient(v[k]);
          if (k * THREADS + tid < n) __stcs(reinterpret_cast<uint4*>(to + k * THREADS * kE), out);
        }
      } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const uint4 out = gradient(v[k]);
          if (k * THREADS + tid < n) store_vec<T>(to + k * THREADS * kE, out, false);
        }
      }
      // the places that the row names are written after the rest, by the warp that has written there
      if (zero) continue;
      if constexpr (has_list(KIND)) {
        const TeacherList list = list_at(lists + static_cast<size_t>(i & 1) * list_bytes(p.K), p.K);
        __syncwarp();
        for (int k = lane; k < result.entries; k += 32) {
          const int column = list.column[k];
          if (!WHOLE && (column < split.head || column >= static_cast<int>(p.V) - split.tail)) continue;  // the closer's
          const unsigned vec = static_cast<unsigned>(column - split.head) / kE - first_vec;
          if (vec % THREADS / 32 == static_cast<unsigned>(warp))
            g[column] = from_float<T>(entry_grad(p, list, k, result.f, result.m, result.inv_s));
        }
      } else if (WHOLE || result.column >= split.head) {
        const int vec = (result.column - split.head) / kE;
        if (vec < split.vecs && vec >= first_vec && vec < first_vec + n && (vec - first_vec) % THREADS == tid)
          g[result.column] = from_float<T>(result.named);
      }
    }
  }
  // the closer's numbers are the CTA's
  __shared__ double all_loss;
  __shared__ int all_rows;
  if (warp == kWarps + 1 && lane == 0) all_loss = loss, all_rows = rows;
  __syncthreads();
  cluster_sync_all();  // no CTA ends while another may still write to its shared memory
  if (aborted)         // pushes that nobody waited for land meanwhile
    for (int i = 0; i < 100; ++i) __nanosleep(1000);
  finish_rows(p, all_loss, all_bits | (aborted ? FLCE_STATUS_BIT_TIMEOUT : 0), all_rows);
}

template <typename T, int KIND, int THREADS, int VPT, int CTAS_PER_SM, bool WHOLE>
cudaError_t launch_parts_of(const RowLossParams& p, PartShape shape, cudaStream_t s) {
  constexpr auto kernel = row_loss_parts_kernel<T, KIND, THREADS, VPT, CTAS_PER_SM, WHOLE>;
  constexpr size_t kLargest = 216 * 1024;  // with what is not dynamic, an SM's shared memory
  const size_t lists = has_list(KIND) ? 2 * list_bytes(p.K) + table_slots(p.K) * 4 : 0;
  const size_t room = kLargest / CTAS_PER_SM - 4096;  // less what is not part_memory
  shape.slot_bytes = (shape.seg_vecs * 16 + 127) & ~127;
  shape.slots = static_cast<int>(room > lists ? (room - lists) / shape.slot_bytes : 1);
  // where gradients are written, one part ahead: with two, more reads among the writes made
  // memory slower (policy loss, bf16 [4096, 128256], 341 -> 328 us; fp32 [1000, 50257] 74 -> 73)
  // (short parts beside lists: two, bf16 [16384, 8192] 131 -> 122 us)
  const int most = p.grad == nullptr ? kPartSlots : has_list(KIND) && shape.slot_bytes <= 16384 ? 2 : 1;
  if (shape.slots > most) shape.slots = most;
  if (shape.slots < 1) shape.slots = 1;
  const size_t smem = static_cast<size_t>(shape.slots) * shape.slot_bytes + lists;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS + 64);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = static_cast<unsigned>(shape.cluster);
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  // clusters that run at a time, by device, CTAs of a row and shared memory: asked for once
  static std::atomic<uint64_t> known[16];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t key = static_cast<uint64_t>(dev + 1) << 48 | static_cast<uint64_t>(smem) << 16;
  uint64_t held = known[shape.cluster].load(std::memory_order_relaxed);
  if ((held & ~uint64_t(0xFFFF)) != key) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLargest));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(shape.cluster));
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    const int most = kRowLossMaxCtas / shape.cluster;
    held = key | static_cast<uint64_t>(clusters < most ? clusters : most);
    known[shape.cluster].store(held, std::memory_order_relaxed);
  }
  const int64_t clusters = static_cast<int64_t>(held & 0xFFFF);
  cfg.gridDim = dim3(static_cast<unsigned>((p.N < clusters ? p.N : clusters) * shape.cluster));
  cfg.numAttrs = p.counts != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, shape);
}

// ---------------------------------------------------------------- host side

template <typename T, int KIND, int THREADS, int VPT, int CTAS_PER_SM>
cudaError_t launch_parts(const RowLossParams& p, const PartShape& shape, cudaStream_t s) {
  constexpr int kE = kVecElems<T>;
  const bool whole = p.V % kE == 0 && aligned_to(p.logits, 16) && p.ld % kE == 0 &&
                     (p.grad == nullptr || (aligned_to(p.grad, 16) && p.ld_grad % kE == 0));
  return whole ? launch_parts_of<T, KIND, THREADS, VPT, CTAS_PER_SM, true>(p, shape, s)
               : launch_parts_of<T, KIND, THREADS, VPT, CTAS_PER_SM, false>(p, shape, s);
}

// Rows of up to 512 vectors (8 KB) by warps (bf16 [32768, 4096] 120 us, by parts 192; of 1024
// vectors, [32768, 8192], 259 and 194); then by parts of up to 2048 vectors (32 KB) by 256
// threads, three CTAs an SM; rows of more than eight of these by parts of up to 4096, two CTAs an SM; and what
// is longer is read twice.  For a teacher's list, which every CTA of a row reads, the larger
// parts from more than four on: bf16 [4096, 128256] 350 -> 325 us (but fp32 [1999, 32001], of
// four parts, 86 -> 94; the policy loss on [4096, 128256] 328 -> 344).  Lists of more than 64
// entries are what takes time themselves: fewest CTAs a row, and kernels of their own, whose
// registers are the list's (bf16 [4096, 32768] with 256 entries 239 -> 130 us, [2048, 128256]
// with 1000 1039 -> 421).
template <typename T, int KIND>
cudaError_t launch_rows_of(const RowLossParams& p, cudaStream_t s) {
  const int64_t vecs = p.V / kVecElems<T>;
  PartShape shape = {};
  if (p.N == 0 || vecs > 8 * 4096) return launch_long<T, KIND>(p, s);
  if (vecs <= 32) return launch_warps<T, KIND, 1>(p, s);
  if (vecs <= 128) return launch_warps<T, KIND, 4>(p, s);
  if (vecs <= 256) return launch_warps<T, KIND, 8>(p, s);
  if (vecs <= 512) return launch_warps<T, KIND, 16>(p, s);
  const bool wide = KIND == kDistillLong ? vecs > 1024 : vecs > (KIND == kDistill ? 4 : 8) * 2048;
  shape.cluster = 1;
  while (div_up(vecs, shape.cluster) > (wide ? 4096 : 2048)) shape.cluster *= 2;
  shape.seg_vecs = static_cast<int>(div_up(vecs, shape.cluster));
  if (shape.seg_vecs <= 1024 && !wide) return launch_parts<T, KIND, 256, 4, 3>(p, shape, s);
  if constexpr (KIND != kDistillLong)
    if (shape.seg_vecs <= 2048 && !wide) return launch_parts<T, KIND, 256, 8, 3>(p, shape, s);
  return launch_parts<T, KIND, 256, 16, 2>(p, shape, s);
}

// All rows of a call: the count that a mean needs first, then the rows.
template <int KIND>
cudaError_t launch_rows(const RowLossParams& given, int dtype, cudaStream_t s) {
  RowLossParams p = given;
  // every CTA counts all rows' targets itself where that is less than a launch takes
  const bool self_count = p.N <= (has_list(KIND) ? 512 : 2048);
  if (p.reduction != FLCE_REDUCTION_MEAN || KIND == kStats || self_count) {
    p.counts = nullptr;
  } else {
    prof_begin(s, FLCE_KERNEL_ROW_COUNT);
    row_count_kernel<KIND><<<kCountCtas, 256, 0, s>>>(p, const_cast<int*>(p.counts));
    const cudaError_t e = cudaGetLastError();
    prof_end(s);
    if (e != cudaSuccess) return e;
  }
  prof_begin(s, FLCE_KERNEL_ROW_LOSS);
  const cudaError_t e = dtype == FLCE_DTYPE_BF16   ? launch_rows_of<__nv_bfloat16, KIND>(p, s)
                        : dtype == FLCE_DTYPE_FP16 ? launch_rows_of<__half, KIND>(p, s)
                                                   : launch_rows_of<float, KIND>(p, s);
  prof_end(s);
  return e;
}

// Workspace of a call over rows: status, arrivals (two, for the calls of two such
// launches), counts, flags, partial losses.
constexpr size_t kRowLossFixed = 512 + kRowLossMaxCtas * (sizeof(int) + sizeof(double));
static_assert(256 + kCountCtas * sizeof(int) <= 512, "counts fit before the flags");

inline void use_workspace(RowLossParams* p, void* workspace, int32_t* status_dev) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->status = status_dev != nullptr ? status_dev : reinterpret_cast<int*>(ws);
  p->own_status = status_dev == nullptr ? 1 : 0;
  p->arrivals = reinterpret_cast<unsigned long long*>(ws + 8);
  p->tag = next_arrival_tag();
  p->counts = reinterpret_cast<const int*>(ws + 256);
  p->flags = reinterpret_cast<int*>(ws + 512);
  p->partial = reinterpret_cast<double*>(ws + 512 + kRowLossMaxCtas * sizeof(int));
  p->timeout_ns = wait_timeout_ns();
}

inline bool row_sizes_ok(int64_t N, int64_t V, int64_t ld) {
  const int64_t most = int64_t(1) << 31;
  return N >= 0 && N < most && V >= 1 && V < most && ld >= V && ld <= (int64_t(1) << 58) / (N > 0 ? N : 1);
}

// What the three losses check alike; `losses`: how many NONE leaves.
inline flce_status_t check_rows(const void* logits, int dtype, int64_t ld, const void* grad, int64_t ld_grad,
                                int64_t N, int64_t V, int64_t losses, int reduction, const float* grad_out,
                                const float* loss, const void* workspace, size_t workspace_bytes, size_t size,
                                const int32_t* status) {
  if (!float_dtype(dtype)) return FLCE_ERR_UNSUPPORTED;
  if (!row_sizes_ok(N, V, ld) || (grad != nullptr && !row_sizes_ok(N, V, ld_grad))) return FLCE_ERR_INVALID_ARG;
  if (reduction < FLCE_REDUCTION_NONE || reduction > FLCE_REDUCTION_MEAN) return FLCE_ERR_INVALID_ARG;
  if (grad_out != nullptr && reduction != FLCE_REDUCTION_NONE) return FLCE_ERR_INVALID_ARG;
  if (N > 0 && logits == nullptr) return FLCE_ERR_INVALID_ARG;
  if (loss == nullptr && (reduction != FLCE_REDUCTION_NONE || losses > 0)) return FLCE_ERR_INVALID_ARG;
  const size_t esz = elem_size(dtype);
  if (!aligned_to(logits, esz) || !aligned_to(grad, esz) || !aligned_to(loss, 4) || !aligned_to(grad_out, 4) ||
      !aligned_to(status, 4))
    return FLCE_ERR_MISALIGNED;
  if (grad != nullptr && N > 0) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(logits), g = reinterpret_cast<uintptr_t>(grad);
    const uintptr_t x_end = x + (static_cast<uintptr_t>(N - 1) * ld + V) * esz;
    const uintptr_t g_end = g + (static_cast<uintptr_t>(N - 1) * ld_grad + V) * esz;
    if (x == g ? (ld != ld_grad && N > 1) : (x < g_end && g < x_end)) return FLCE_ERR_INVALID_ARG;
  }
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < size) return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

inline RowLossParams row_params(const void* logits, int64_t ld, void* grad, int64_t ld_grad, int64_t N, int64_t V,
                                int reduction, float grad_scale, const float* grad_out, float* loss,
                                float temperature) {
  RowLossParams p = {};
  p.logits = logits, p.ld = ld, p.grad = grad, p.ld_grad = ld_grad, p.N = N, p.V = V;
  p.reduction = reduction, p.grad_scale = grad_scale, p.grad_out = grad_out;
  p.loss_rows = reduction == FLCE_REDUCTION_NONE ? loss : nullptr;
  p.loss = reduction == FLCE_REDUCTION_NONE ? nullptr : loss;
  p.temperature = temperature, p.inv_t = 1.f / temperature;
  p.c = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
  return p;
}

inline bool positive(float x) { return x > 0.f && x <= 3.402823466e38f; }
// Temperatures: T, 1 / T and T^2 times a loss stay in the range of fp32.
inline bool temperature_ok(float t) { return t >= 1e-4f && t <= 1e4f; }

}  // namespace
}  // namespace flce
