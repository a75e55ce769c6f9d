// Rows of a table by token, and the table's gradient.
//
// Forward is a gather: memory moves N rows once each way.
//
// Backward adds up the rows of grad_y that belong to one id.  Additions in the order in
// which CTAs come (atomics on the table) would change the result from run to run, so the
// tokens are sorted by id first, stably, and the sorted list is cut into tiles of kTile
// tokens whatever their ids are: a frequent id (padding, a newline) then costs no more
// than many rare ones.  A tile writes the sums of ids that lie within it; of an id that
// goes on in the next tile it leaves a partial row, and a last kernel adds those up.
#include <algorithm>
#include <atomic>

#include "elem.cuh"
#include "ptx.cuh"

namespace flce {
namespace {

__device__ __forceinline__ int64_t id_at(const void* ids, int ids32, int64_t i) {
  return ids32 ? __ldg(static_cast<const int32_t*>(ids) + i) : __ldg(static_cast<const int64_t*>(ids) + i);
}

// N elements of one type in a vector of 16 bytes, or one element.
template <typename T, int E>
struct alignas(E == 1 ? alignof(T) : 16) Elems {
  T v[E];
};

// ---------------------------------------------------------------- forward

struct LookupParams {
  const void* table;
  const void* ids;
  void* y;
  int64_t ld_table, ld_y, N, V, H;
  int64_t parts;  // of a row, of 32 * kLookupUnroll vectors each
  int ids32;
  float scale;
  int* status;
};

constexpr int kLookupUnroll = 4;
constexpr int kLookupWarps = 4;

// A part of a row by each warp, of rows that are whole vectors.
template <typename T>
__global__ void __launch_bounds__(32 * kLookupWarps) embedding_kernel(const LookupParams p) {
  constexpr int E = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kLookupWarps + (threadIdx.x >> 5); item < p.N * p.parts;
       item += static_cast<int64_t>(gridDim.x) * kLookupWarps) {
    const int64_t n = item / p.parts, part = item % p.parts;
    const int64_t id = id_at(p.ids, p.ids32, n);
    const bool inside = id >= 0 && id < p.V;
    if (!inside && p.status != nullptr && lane == 0 && part == 0) atomicOr(p.status, FLCE_STATUS_BIT_TARGET_RANGE);
    const T* from = static_cast<const T*>(p.table) + (inside ? id : 0) * p.ld_table;
    T* to = static_cast<T*>(p.y) + n * p.ld_y;
    const int64_t first = (part * 32 * kLookupUnroll + lane) * E;
    Elems<T, E> v[kLookupUnroll];
#pragma unroll
    for (int i = 0; i < kLookupUnroll; ++i) {
      const int64_t at = first + i * 32 * E;
      if (at < p.H && inside) v[i] = *reinterpret_cast<const Elems<T, E>*>(from + at);
    }
#pragma unroll
    for (int i = 0; i < kLookupUnroll; ++i) {
      const int64_t at = first + i * 32 * E;
      if (at >= p.H) break;
#pragma unroll
      for (int k = 0; k < E; ++k) v[i].v[k] = from_float<T>(inside ? to_float(v[i].v[k]) * p.scale : 0.f);
      // past the caches, which keep the table's rows for the next token of the id (37.7 -> 31.0 us)
      __stcs(reinterpret_cast<uint4*>(to + at), *reinterpret_cast<const uint4*>(&v[i]));
    }
  }
}

// The 16 bytes that start `from` bytes (0 to 15, a multiple of 2) into two vectors.
__device__ __forceinline__ uint4 across(const uint4& a, const uint4& b, unsigned from) {
  const unsigned bits = (from & 3) * 8;
  const auto shifted = [&](uint32_t v, uint32_t w, uint32_t x, uint32_t y, uint32_t z) {
    return make_uint4(__funnelshift_r(v, w, bits), __funnelshift_r(w, x, bits), __funnelshift_r(x, y, bits),
                      __funnelshift_r(y, z, bits));
  };
  switch (from >> 2) {  // the same for a whole row
    case 0: return shifted(a.x, a.y, a.z, a.w, b.x);
    case 1: return shifted(a.y, a.z, a.w, b.x, b.y);
    case 2: return shifted(a.z, a.w, b.x, b.y, b.z);
    default: return shifted(a.w, b.x, b.y, b.z, b.w);
  }
}

// Rows that start anywhere: vectors by the places of y's row, each made of the two vectors of
// the table's row that it lies across; what has no two such vectors within the row goes by
// elements, at both ends.  (By elements alone bf16 [16384, 4095] took 86 us.)
template <typename T>
__global__ void __launch_bounds__(32 * kLookupWarps) embedding_shifted_kernel(const LookupParams p) {
  constexpr int kE = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const int bytes = static_cast<int>(p.H * sizeof(T));
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kLookupWarps + (threadIdx.x >> 5); item < p.N * p.parts;
       item += static_cast<int64_t>(gridDim.x) * kLookupWarps) {
    const int64_t n = item / p.parts;
    const int part = static_cast<int>(item % p.parts);
    const int64_t id = id_at(p.ids, p.ids32, n);
    const bool inside = id >= 0 && id < p.V;
    if (!inside && p.status != nullptr && lane == 0 && part == 0) atomicOr(p.status, FLCE_STATUS_BIT_TARGET_RANGE);
    const T* from = static_cast<const T*>(p.table) + (inside ? id : 0) * p.ld_table;
    T* to = static_cast<T*>(p.y) + n * p.ld_y;
    // vector j is y's bytes head + 16 j on; it starts `shift` bytes into a vector of the table
    const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(to) & 15)) & 15);
    const unsigned shift = static_cast<unsigned>(reinterpret_cast<uintptr_t>(from) + head) & 15;
    const int vecs = bytes > head ? (bytes - head) / 16 : 0;
    const int first = static_cast<int>(shift) > head ? 1 : 0;
    int end = vecs;
    if (shift != 0) {
      const int room = bytes - head + static_cast<int>(shift) - 16;  // from vector 0's first part on, less one vector
      end = room >= 16 ? min(vecs, room / 16) : 0;
    }
    if (end < first) end = first;
    const uint4* source = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(from) + head - shift);
    uint4* target = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(to) + head);
    uint4 a[kLookupUnroll], b[kLookupUnroll];
    const int j0 = part * 32 * kLookupUnroll + lane;
#pragma unroll
    for (int i = 0; i < kLookupUnroll; ++i) {
      const int j = j0 + i * 32;
      if (j < first || j >= end || !inside) continue;
      a[i] = __ldg(source + j);
      b[i] = shift != 0 ? __ldg(source + j + 1) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kLookupUnroll; ++i) {
      const int j = j0 + i * 32;
      if (j < first || j >= end) continue;
      uint4 v = inside ? across(a[i], b[i], shift) : make_uint4(0, 0, 0, 0);
      T* e = reinterpret_cast<T*>(&v);
#pragma unroll
      for (int k = 0; k < kE; ++k) e[k] = from_float<T>(inside ? to_float(e[k]) * p.scale : 0.f);
      __stcs(target + j, v);
    }
    if (part != 0) continue;
    const int before = min((head + 16 * first) / static_cast<int>(sizeof(T)), static_cast<int>(p.H));
    const int after = min(max(before, (head + 16 * end) / static_cast<int>(sizeof(T))), static_cast<int>(p.H));
    for (int h = lane; h < before + static_cast<int>(p.H) - after; h += 32) {
      const int at = h < before ? h : after + h - before;
      to[at] = from_float<T>(inside ? to_float(from[at]) * p.scale : 0.f);
    }
  }
}

template <typename T>
cudaError_t lookup(LookupParams p, cudaStream_t s) {
  constexpr int kE = 16 / sizeof(T);
  const bool vectors = aligned_to(p.table, 16) && aligned_to(p.y, 16) && p.H % kE == 0 &&
                       (p.ld_table % kE == 0 || p.V == 1) && (p.ld_y % kE == 0 || p.N == 1);
  p.parts = div_up(p.H, 32 * kLookupUnroll * kE);
  const int64_t ctas = div_up(p.N * p.parts, kLookupWarps), most = int64_t(1) << 30;
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  prof_begin(s, FLCE_KERNEL_EMBEDDING);
  if (vectors)
    embedding_kernel<T><<<grid, 32 * kLookupWarps, 0, s>>>(p);
  else
    embedding_shifted_kernel<T><<<grid, 32 * kLookupWarps, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  prof_end(s);
  return e;
}

// ---------------------------------------------------------------- sorting tokens by id

struct SortParams {
  const void* ids;
  int ids32;
  int N, V;            // keys are ids, or V for tokens that add nothing
  int64_t padding;
  int passes, digit;   // bits of a pass
  int room;            // places of a CTA in shared memory
  int* keys[2];        // [N] each; the result is in keys[0], tokens[0]
  int* tokens[2];
  uint32_t* hit;       // a bit for each row of the table that gets something, or null
  int* status;
};

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortDigit = 9;       // most bits of a pass: two passes reach 2^18 ids
constexpr int kSortRoom = 8192;     // most tokens that a CTA holds in shared memory
constexpr int kSortCtas = 8;        // of a cluster
constexpr int kSortAlone = 2048;    // most tokens that one CTA sorts without a cluster

__device__ __forceinline__ void store_cluster_u64(uint32_t at, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void store_cluster_s32(uint32_t at, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

constexpr int kSortEach = kSortRoom / kSortThreads;  // a thread's tokens at most

// Stable radix sort, least significant digit first, by one CTA or one cluster.  Each warp
// owns a stretch of the list: it counts its digits, the counts are added up over warps and
// CTAs, and it puts its keys where those before them leave room.  Lanes with the same digit
// find one another by match.  SHARED: a pass has its stretch in registers, with each token's
// place among those of its digit, and the list is in shared memory from pass to pass, each
// place in the CTA that reads it next.  Longer lists go through global memory.
template <int CTAS, bool SHARED>
__global__ void __launch_bounds__(kSortThreads) token_sort_kernel(const SortParams p) {
  extern __shared__ __align__(16) uint8_t sort_memory[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << p.digit;
  int* counts = reinterpret_cast<int*>(sort_memory);  // [warps][digits]
  int* totals = counts + kSortWarps * digits;         // [CTAs][digits], by the CTA that has them
  int* starts = totals + CTAS * digits;               // [digits]
  uint64_t* list = reinterpret_cast<uint64_t*>(starts + digits);  // [room]: tokens above, keys below
  int* own = counts + warp * digits;
  __shared__ int warp_sums[32];
  const int rank = CTAS > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
  if (CTAS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int64_t warps = static_cast<int64_t>(CTAS) * kSortWarps;
  const int64_t stretch = (p.N + warps * 32 - 1) / (warps * 32) * 32;
  const int64_t cta_from = rank * kSortWarps * stretch;
  const int64_t from = cta_from + warp * stretch;
  const int64_t to = from + stretch < p.N ? from + stretch : p.N;
  int bits = 0;
  if (p.hit != nullptr)
    for (int i = rank * kSortThreads + threadIdx.x; i < (p.V + 31) / 32; i += CTAS * kSortThreads) p.hit[i] = 0;
  const auto first_entry = [&](int64_t i) -> uint64_t {
    const int64_t id = id_at(p.ids, p.ids32, i);
    const bool inside = id >= 0 && id < p.V;
    if (!inside) bits |= FLCE_STATUS_BIT_TARGET_RANGE;
    return static_cast<uint64_t>(i) << 32 | static_cast<uint32_t>(!inside || id == p.padding ? p.V : id);
  };
  // frequent ids would queue up at their word
  const auto set_hit = [&](int key) {
    if (key < p.V && !(__ldcg(p.hit + (key >> 5)) >> (key & 31) & 1)) atomicOr(p.hit + (key >> 5), 1u << (key & 31));
  };
  uint64_t held[SHARED ? kSortEach : 1];  // entries of a pass, and their places among the warp's of that digit
  int place[SHARED ? kSortEach : 1];
  if constexpr (SHARED) {
#pragma unroll
    for (int j = 0; j < kSortEach; ++j) {
      const int64_t i = from + j * 32 + lane;
      held[j] = i < to ? first_entry(i) : 0;
    }
  }
  if (CTAS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA runs
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit;
    const bool last = pass == p.passes - 1;
    // in global memory the passes go to and fro, and the last one ends in array 0
    const bool to_first = ((p.passes - 1 - pass) & 1) == 0;
    int* const keys_to = to_first ? p.keys[0] : p.keys[1];
    int* const tokens_to = to_first ? p.tokens[0] : p.tokens[1];
    const int* const keys_from = to_first ? p.keys[1] : p.keys[0];
    const int* const tokens_from = to_first ? p.tokens[1] : p.tokens[0];
    const auto entry = [&](int64_t i) -> uint64_t {
      if (pass == 0) return first_entry(i);
      return static_cast<uint64_t>(__ldcg(tokens_from + i)) << 32 | static_cast<uint32_t>(__ldcg(keys_from + i));
    };
    const auto digit_of = [&](uint64_t e) { return static_cast<int>(static_cast<uint32_t>(e) >> shift) & (digits - 1); };
    for (int d = lane; d < digits; d += 32) own[d] = 0;
    __syncwarp();
    if constexpr (SHARED) {
      if (pass > 0) {
#pragma unroll
        for (int j = 0; j < kSortEach; ++j) {
          const int64_t i = from + j * 32 + lane;
          if (i < to) held[j] = list[i - cta_from];
        }
      }
#pragma unroll
      for (int j = 0; j < kSortEach; ++j) {
        if (from + j * 32 >= to) break;
        const bool valid = from + j * 32 + lane < to;
        const int d = valid ? digit_of(held[j]) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        place[j] = valid ? own[d] + __popc(same & ((1u << lane) - 1)) : 0;
        __syncwarp();
        if (valid && lane == __ffs(same) - 1) own[d] += __popc(same);
        __syncwarp();
      }
    } else {
      for (int64_t i0 = from; i0 < to; i0 += 32) {
        const bool valid = i0 + lane < to;
        const int d = valid ? digit_of(entry(i0 + lane)) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (valid && lane == __ffs(same) - 1) own[d] += __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
    // counts of the CTA's warps become those before each; every CTA gets this one's totals
    for (int d = threadIdx.x; d < digits; d += kSortThreads) {
      int sum = 0;
#pragma unroll
      for (int w0 = 0; w0 < kSortWarps; w0 += 16) {
        int c[16];  // read before any is written: the compiler cannot tell the words apart
#pragma unroll
        for (int w = 0; w < 16; ++w) c[w] = counts[(w0 + w) * digits + d];
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          counts[(w0 + w) * digits + d] = sum;
          sum += c[w];
        }
      }
      if (CTAS == 1) totals[d] = sum;
#pragma unroll
      for (int r = 0; r < CTAS && CTAS > 1; ++r)
        store_cluster_s32(map_to_cta(smem_addr(totals + rank * digits + d), r), sum);
    }
    // (and the bits of `hit` are cleared, before any CTA sets one; all have read their part of `list`)
    if (CTAS > 1)
      cluster_sync_all();
    else
      __syncthreads();
    // where a digit's keys start: after all smaller digits, and those of the CTAs before
    int before = 0, all = 0;
    const int d = threadIdx.x;  // digits <= threads
    if (d < digits) {
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
        const int c = totals[r * digits + d];
        if (r < rank) before += c;
        all += c;
      }
    }
    int scan = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += up;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    int sum = lane < warp ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (d < digits) starts[d] = scan - all + before + sum;
    __syncthreads();
    if constexpr (SHARED) {
#pragma unroll
      for (int j = 0; j < kSortEach; ++j) {
        const int64_t i = from + j * 32 + lane;
        if (i >= to) break;
        const uint64_t e = held[j];
        const int digit = digit_of(e), at = starts[digit] + own[digit] + place[j];
        if (last) {
          p.keys[0][at] = static_cast<int>(e);
          p.tokens[0][at] = static_cast<int>(e >> 32);
        } else if (CTAS == 1) {
          list[at] = e;
        } else {
          const unsigned cta = static_cast<unsigned>(at) / static_cast<unsigned>(p.room);
          store_cluster_u64(map_to_cta(smem_addr(list + (at - cta * p.room)), cta), e);
        }
      }
      if (pass == 0 && p.hit != nullptr) {
#pragma unroll
        for (int j = 0; j < kSortEach; ++j)
          if (from + j * 32 + lane < to) set_hit(static_cast<int>(held[j]));
      }
    } else {
      for (int64_t i0 = from; i0 < to; i0 += 32) {
        const bool valid = i0 + lane < to;
        const uint64_t e = valid ? entry(i0 + lane) : 0;
        const int digit = valid ? digit_of(e) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        int at = 0;
        if (valid) at = starts[digit] + own[digit] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (valid && lane == __ffs(same) - 1) own[digit] += __popc(same);
        if (valid) {
          keys_to[at] = static_cast<int>(e);
          tokens_to[at] = static_cast<int>(e >> 32);
          if (pass == 0 && p.hit != nullptr) set_hit(static_cast<int>(e));
        }
        __syncwarp();
      }
    }
    // the keys are in place, and the totals have been read; after the last pass nobody looks
    if (CTAS == 1)
      __syncthreads();
    else if (!last)
      cluster_sync_all();
  }
  if (bits != 0 && p.status != nullptr) atomicOr(p.status, bits);
}

// ---------------------------------------------------------------- sums

constexpr int kTile = 32;          // sorted tokens of a tile: one a lane
constexpr int kSumWarps = 4;
constexpr int kAhead = 8;          // tokens whose rows are loaded at a time, by elements
constexpr int kRing = 16;          // tokens whose rows are on their way, by vectors
constexpr int kRingStep = 4;       // of them at a time

struct SumParams {
  const void* grad_y;
  int64_t ld, H;
  int N, V;
  const int* keys;
  const int* tokens;
  const uint32_t* hit;  // null: rows without tokens are not written
  float* table;
  float* partial;       // [tiles][2][H]: of an id that began before a tile, and of one that goes on after it
  int* joins;           // [tiles]: whether an id begins in it that goes on past the next one
  int accumulate;
  float scale;
  int tiles, columns;   // tiles, and pieces of a row, each a warp's
  unsigned zero_ctas;   // the grid's first, which write zeros
  // without sorting
  const void* ids;
  int ids32;
  int64_t padding;
  int* status;
};

__device__ __forceinline__ void write_zeros(float* row, int64_t H, int lane, bool vectors) {
  if (vectors) {
    for (int64_t h = lane * 4; h < H; h += 128) __stcs(reinterpret_cast<float4*>(row + h), make_float4(0, 0, 0, 0));
  } else {
    for (int64_t h = lane; h < H; h += 32) __stcs(row + h, 0.f);
  }
}

// A read that stays where it is written, so that several are on their way before the first
// is waited for (the compiler would move each to its use: 8 rows one after another took
// 5700 cycles a warp).
template <typename T, int E>
__device__ __forceinline__ Elems<T, E> load_now(const T* p) {
  Elems<T, E> r;
  if constexpr (E > 1) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    r = *reinterpret_cast<const Elems<T, E>*>(&v);
  } else if constexpr (sizeof(T) == 4) {
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(*reinterpret_cast<float*>(&r.v[0])) : "l"(p));
  } else {
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(*reinterpret_cast<uint16_t*>(&r.v[0])) : "l"(p));
  }
  return r;
}

// A lane's columns of one row: GROUPS times E, 32 * E apart.  `at`: where they are in any
// row; a lane past the row's end reads the row's last columns.
template <typename T, int E, int GROUPS>
struct Columns {
  Elems<T, E> v[GROUPS];
  __device__ __forceinline__ void load(const T* row, const int (&at)[GROUPS]) {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) v[g] = load_now<T, E>(row + at[g]);
  }
};
template <int E, int GROUPS>
__device__ __forceinline__ void columns_at(int64_t first, int64_t H, int (&at)[GROUPS]) {
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const int64_t h = first + g * 32 * E;
    at[g] = static_cast<int>(h < H ? h : H - E);
  }
}

template <int E, int GROUPS>
struct Sums {
  float s[GROUPS][E];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
      for (int k = 0; k < E; ++k) s[g][k] = 0.f;
  }
  template <typename T>
  __device__ __forceinline__ void add(const Columns<T, E, GROUPS>& c) {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
      for (int k = 0; k < E; ++k) s[g][k] += to_float(c.v[g].v[k]);
  }
  // To a row of fp32, times `scale`; `add`: by the memory system, which nothing waits for
  // (an element gets one such addition in a call, so that their order is no matter).
  __device__ __forceinline__ void store(float* row, int64_t first, int64_t H, float scale, bool add) const {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int64_t h = first + g * 32 * E;
      if (h >= H) break;
      if constexpr (E > 1) {
#pragma unroll
        for (int q = 0; q < E; q += 4) {
          const float4 o = make_float4(s[g][q] * scale, s[g][q + 1] * scale, s[g][q + 2] * scale, s[g][q + 3] * scale);
          float4* at = reinterpret_cast<float4*>(row + h + q);
          if (add)
            red_add_f32x4(at, o);
          else
            *at = o;
        }
      } else {
        if (add)
          atomicAdd(row + h, s[g][0] * scale);
        else
          row[h] = s[g][0] * scale;
      }
    }
  }
};

__device__ __forceinline__ void copy_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

// One tile's columns by each warp: a lane holds the tile's keys and those of the next one,
// and all go through the tokens in order, kAhead rows on their way.  An id that ends in the
// next tile is finished by the tile in which it begins, so that partial rows are left for
// ids of more than kTile tokens alone.
template <typename T, int E, int GROUPS>
__global__ void __launch_bounds__(32 * kSumWarps, 6) embedding_sum_kernel(const SumParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  if (blockIdx.x < p.zero_ctas) {
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * kSumWarps + warp; v < p.V; v += p.zero_ctas * kSumWarps)
      if (!(__ldg(p.hit + (v >> 5)) >> (v & 31) & 1)) write_zeros(p.table + v * p.H, p.H, lane, E > 1);
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x - p.zero_ctas) * kSumWarps + warp;
  if (item >= static_cast<int64_t>(p.tiles) * p.columns) return;
  const int tile = static_cast<int>(item / p.columns), column = static_cast<int>(item % p.columns);
  const int64_t begin = static_cast<int64_t>(tile) * kTile;
  const auto key_at = [&](int64_t i) { return i >= 0 && i < p.N ? __ldg(p.keys + i) : -1; };
  const int k0 = key_at(begin + lane), k1 = key_at(begin + kTile + lane);
  const int token0 = begin + lane < p.N ? __ldg(p.tokens + begin + lane) : 0;
  const int token1 = begin + kTile + lane < p.N ? __ldg(p.tokens + begin + kTile + lane) : 0;
  // neighbours: the key before this tile, before the tile before, and after the next one
  const int around = key_at(lane == 0 ? begin - 1 : lane == 1 ? begin - 1 - kTile : begin + 2 * kTile);
  const int before = __shfl_sync(0xffffffffu, around, 0), long_before = __shfl_sync(0xffffffffu, around, 1);
  const int after = __shfl_sync(0xffffffffu, around, 2);
  const int head = __shfl_sync(0xffffffffu, k0, 0), tail = __shfl_sync(0xffffffffu, k0, kTile - 1);
  const int next = __shfl_sync(0xffffffffu, k1, 0);
  // bit i: token i is its id's last one (places beyond the list, and tokens that add
  // nothing, have keys of -1 and V and end it)
  int up = __shfl_down_sync(0xffffffffu, k0, 1);
  const unsigned ends0 = __ballot_sync(0xffffffffu, k0 != (lane == 31 ? next : up));
  up = __shfl_down_sync(0xffffffffu, k1, 1);
  const unsigned ends1 = __ballot_sync(0xffffffffu, k1 != (lane == 31 ? after : up));
  const unsigned used0 = __ballot_sync(0xffffffffu, k0 >= 0 && k0 < p.V);
  int to = __popc(used0);  // tokens of this tile (they come first)
  if (to == 0) {
    if (column == 0 && lane == 0) p.joins[tile] = 0;
    return;
  }
  int from = 0;
  bool head_partial = false, tail_partial = false;
  if (before == head) {
    // the id began before: the tile before has finished it if it began there and ends here
    const bool ends_here = ends0 != 0;
    if (long_before != head && ends_here)
      from = __ffs(ends0);
    else
      head_partial = true;
  }
  const bool one_id = ends0 == 0;  // and it goes on
  if (to == kTile && next == tail && !(one_id && before == head)) {
    if (ends1 != 0)
      to += __ffs(ends1);          // ends in the next tile
    else
      tail_partial = true;
  }
  if (column == 0 && lane == 0) p.joins[tile] = tail_partial;
  if (from >= to) return;
  const uint64_t ends = static_cast<uint64_t>(ends1) << 32 | ends0;
  const int64_t first = (static_cast<int64_t>(column) * GROUPS * 32 + lane) * E;
  const T* rows = static_cast<const T*>(p.grad_y);
  int at[GROUPS];
  columns_at<E, GROUPS>(first, p.H, at);
  Sums<E, GROUPS> sum;
  sum.clear();
  float* const partial = p.partial + static_cast<int64_t>(tile) * 2 * p.H;
  const auto add = [&](int t, const Columns<T, E, GROUPS>& row) {
    sum.add(row);
    if (!(ends >> t & 1)) return;
    if (head_partial) {
      sum.store(partial, first, p.H, 1.f, false);
      head_partial = false;
    } else {
      const int key = __shfl_sync(0xffffffffu, t < kTile ? k0 : k1, t & 31);
      sum.store(p.table + key * p.H, first, p.H, p.scale, p.accumulate != 0);
    }
    sum.clear();
  };
  const auto token_at = [&](int t) -> int64_t { return __shfl_sync(0xffffffffu, t < kTile ? token0 : token1, t & 31); };
  if constexpr (E > 1) {
    // each lane's vectors of the next kRing tokens are on their way into its own places of shared memory
    extern __shared__ __align__(16) uint4 ring_memory[];
    uint4* const ring = ring_memory + warp * kRing * 32 + lane;
    const auto fetch = [&](int t) {
#pragma unroll
      for (int a = 0; a < kRingStep; ++a) {
        const int64_t n = token_at(t + a < to ? t + a : to - 1);
        if (t + a < to) copy_async(ring + (t + a - from) % kRing * 32, rows + n * p.ld + at[0]);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int g = 0; g < kRing / kRingStep; ++g) fetch(from + g * kRingStep);
    for (int t0 = from; t0 < to; t0 += kRingStep) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing / kRingStep - 1) : "memory");
      Columns<T, E, GROUPS> held[kRingStep];
#pragma unroll
      for (int a = 0; a < kRingStep; ++a)
        held[a].v[0] = *reinterpret_cast<const Elems<T, E>*>(ring + (t0 + a - from) % kRing * 32);
#pragma unroll
      for (int a = 0; a < kRingStep; ++a)
        if (t0 + a < to) add(t0 + a, held[a]);
      fetch(t0 + kRing);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    Columns<T, E, GROUPS> held[kAhead];
    for (int t0 = from; t0 < to; t0 += kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a)  // past the end: the last one again
        held[a].load(rows + token_at(t0 + a < to ? t0 + a : to - 1) * p.ld, at);
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (t0 + a < to) add(t0 + a, held[a]);
    }
  }
  if (head_partial)  // one id, that goes on
    sum.store(partial, first, p.H, 1.f, false);
  else if (tail_partial)
    sum.store(partial + p.H, first, p.H, 1.f, false);
}

constexpr int kJoinWarps = 8;
constexpr int kJoinTiles = 8;
constexpr int kJoinBatch = 64;

// Adds up the partial rows of ids that begin in a tile and go on past the next one, in the
// order of the tiles: each warp a stretch of them by batches, then the warps' sums, so that no
// chain of additions is long (3 * 2^20 equal rows of one id, without batches: off by 1e-4 of
// the sum).  A CTA has 32 * E columns and looks for such ids in kJoinTiles tiles at a time,
// one a lane.
template <int E>
__global__ void __launch_bounds__(32 * kJoinWarps) embedding_join_kernel(const SumParams p) {
  using Part = Elems<float, E>;
  __shared__ Part sums[kJoinWarps][32];
  __shared__ int last_tile;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t h = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * E;
  const auto key_at = [&](int64_t i) { return i >= 0 && i < p.N ? __ldg(p.keys + i) : -1; };
  for (int tile0 = blockIdx.x * kJoinTiles; tile0 < p.tiles; tile0 += gridDim.x * kJoinTiles) {
    const bool joins = lane < kJoinTiles && tile0 + lane < p.tiles && __ldg(p.joins + tile0 + lane) != 0;
    unsigned left = __ballot_sync(0xffffffffu, joins);
    while (left != 0) {  // the same in every warp
      const int tile = tile0 + __ffs(left) - 1;
      left &= left - 1;
      const int key = key_at(static_cast<int64_t>(tile) * kTile + kTile - 1);
      // the tile in which the id ends: the first whose last key is another
      if (threadIdx.x == 0) last_tile = p.tiles - 1;
      __syncthreads();
      for (int t0 = tile + 1;; t0 += 32 * kJoinWarps) {
        const int t = t0 + threadIdx.x;
        const bool ends = t >= p.tiles - 1 || key_at(static_cast<int64_t>(t) * kTile + kTile) != key;
        if (ends && t < p.tiles) atomicMin(&last_tile, t);
        if (__syncthreads_or(ends)) break;
      }
      const int parts = last_tile - tile + 1, each = (parts + kJoinWarps - 1) / kJoinWarps;
      Part sum = {};
      if (h < p.H) {
        const int to = (warp + 1) * each < parts ? (warp + 1) * each : parts;
        for (int i0 = warp * each; i0 < to; i0 += kJoinBatch) {
          Part batch = {};
          const int end = i0 + kJoinBatch < to ? i0 + kJoinBatch : to;
#pragma unroll 8
          for (int i = i0; i < end; ++i) {
            const Part v =
                *reinterpret_cast<const Part*>(p.partial + (static_cast<int64_t>(tile + i) * 2 + (i == 0)) * p.H + h);
#pragma unroll
            for (int k = 0; k < E; ++k) batch.v[k] += v.v[k];
          }
#pragma unroll
          for (int k = 0; k < E; ++k) sum.v[k] += batch.v[k];
        }
      }
      sums[warp][lane] = sum;
      __syncthreads();
      if (warp == 0 && h < p.H) {
        Part* at = reinterpret_cast<Part*>(p.table + key * p.H + h);
        Part out = {};
        if (p.accumulate) out = *at;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          float total = 0.f;
#pragma unroll
          for (int w = 0; w < kJoinWarps; ++w) total += sums[w][lane].v[k];
          out.v[k] += total * p.scale;
        }
        *at = out;
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- few tokens

constexpr int kFewTokens = 1024;
constexpr int kFewCtas = 8192;      // most CTAs that compare an id with all others
constexpr int kFewWarps = 4;
constexpr int kFewZeroRows = 32;    // rows of the table that a CTA looks after,
constexpr int kFewZeroColumns = 2048;  // and so many of their columns

// Without sorting, in one launch: a CTA for each token and piece of a row compares the
// token's id with all others; the first token of an id adds up its rows, each warp every
// kFewWarps-th one of them, and then the warps' sums.  The CTAs before those write zeros to
// rows that no token has.
template <typename T, int E, int GROUPS>
__global__ void __launch_bounds__(32 * kFewWarps) embedding_few_kernel(const SumParams p) {
  __shared__ unsigned match[kFewTokens / 32];
  __shared__ unsigned hit;
  __shared__ Sums<E, GROUPS> sums[kFewWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto key_of = [&](int i) -> int64_t {
    const int64_t id = i < p.N ? id_at(p.ids, p.ids32, i) : -1;
    return id == p.padding || id >= p.V ? -1 : id;
  };
  if (blockIdx.x < p.zero_ctas) {
    const unsigned pieces = static_cast<unsigned>((p.H + kFewZeroColumns - 1) / kFewZeroColumns);
    const int64_t v0 = static_cast<int64_t>(blockIdx.x / pieces) * kFewZeroRows;
    const int64_t h0 = static_cast<int64_t>(blockIdx.x % pieces) * kFewZeroColumns;
    if (threadIdx.x == 0) hit = 0;
    __syncthreads();
    unsigned mine = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.N; i += 32 * kFewWarps) {
      const int64_t at = key_of(i) - v0;
      if (at >= 0 && at < kFewZeroRows) mine |= 1u << at;
    }
    if (mine != 0) atomicOr(&hit, mine);
    __syncthreads();
    for (int r = warp; r < kFewZeroRows && v0 + r < p.V; r += kFewWarps)
      if (!(hit >> r & 1))
        write_zeros(p.table + (v0 + r) * p.H + h0, p.H - h0 < kFewZeroColumns ? p.H - h0 : kFewZeroColumns, lane, E > 1);
    return;
  }
  const int n = (blockIdx.x - p.zero_ctas) / p.columns, column = (blockIdx.x - p.zero_ctas) % p.columns;
  const int64_t key = key_of(n);
  if (p.status != nullptr && column == 0 && threadIdx.x == 0) {
    const int64_t id = id_at(p.ids, p.ids32, n);
    if (id < 0 || id >= p.V) atomicOr(p.status, FLCE_STATUS_BIT_TARGET_RANGE);
  }
  if (key < 0) return;
  const int words = (p.N + 31) / 32;
  for (int w = warp; w < words; w += kFewWarps) {
    const unsigned same = __ballot_sync(0xffffffffu, key_of(w * 32 + lane) == key);
    if (lane == 0) match[w] = same;
  }
  __syncthreads();
  // an earlier token of the id?  (the first word that has one decides, for all lanes)
  for (int w = 0; w <= n / 32; ++w) {
    const unsigned earlier = w == n / 32 ? match[w] & ((1u << (n & 31)) - 1) : match[w];
    if (earlier != 0) return;
  }
  const int64_t first = (static_cast<int64_t>(column) * GROUPS * 32 + lane) * E;
  const T* rows = static_cast<const T*>(p.grad_y);
  Sums<E, GROUPS> sum;
  sum.clear();
  int at[GROUPS];
  columns_at<E, GROUPS>(first, p.H, at);
  int count = 0;  // tokens of the id so far
  constexpr int kFewAhead = 4;
  Columns<T, E, GROUPS> held[kFewAhead];
  int holding = 0;
  for (int w = n / 32; w < words; ++w) {
    for (unsigned m = match[w]; m != 0; m &= m - 1, ++count) {
      if (count % kFewWarps != warp) continue;
      const int64_t t = w * 32 + __ffs(m) - 1;
#pragma unroll
      for (int a = 0; a < kFewAhead; ++a)
        if (a == holding) held[a].load(rows + t * p.ld, at);
      if (++holding == kFewAhead) {
#pragma unroll
        for (int a = 0; a < kFewAhead; ++a) sum.add(held[a]);
        holding = 0;
      }
    }
  }
#pragma unroll
  for (int a = 0; a < kFewAhead; ++a)
    if (a < holding) sum.add(held[a]);
  if (count > 1) {
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kFewWarps; ++w)
#pragma unroll
      for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int k = 0; k < E; ++k) sum.s[g][k] += sums[w][lane].s[g][k];
  } else if (warp != 0) {
    return;
  }
  sum.store(p.table + key * p.H, first, p.H, p.scale, p.accumulate != 0);
}

// Whether the launches hold the tiles' pieces of a row (whether they go by vectors or not)
// and the join's columns, 32 a CTA: 65535 of these.
bool launches_hold(int64_t N, int64_t H) {
  return div_up(div_up(N, kTile) * div_up(H, 128), kSumWarps) + 8 * 1024 < (int64_t(1) << 31) && div_up(H, 32) <= 65535;
}

struct EmbeddingLayout {
  size_t keys[2], tokens[2], hit, joins, partial, total;
};

bool embedding_layout(int64_t N, int64_t V, int64_t H, EmbeddingLayout* at) {
  if (N < 0 || N >= (int64_t(1) << 31) - kTile || V < 1 || V >= (int64_t(1) << 31) - 1 || H < 1 || H >= (1 << 24))
    return false;
  const size_t list = align_up(static_cast<size_t>(N) * 4, 256);
  at->keys[0] = 0, at->keys[1] = list, at->tokens[0] = 2 * list, at->tokens[1] = 3 * list;
  at->hit = 4 * list;
  at->joins = align_up(at->hit + static_cast<size_t>(div_up(V, 32)) * 4, 256);
  at->partial = align_up(at->joins + static_cast<size_t>(div_up(N, kTile)) * 4, 256);
  at->total = align_up(at->partial + static_cast<size_t>(div_up(N, kTile)) * 2 * H * 4, 256);
  return true;
}

template <int CTAS, bool SHARED>
cudaError_t launch_sort(SortParams p, cudaStream_t s) {
  p.room = SHARED ? static_cast<int>(div_up(p.N, CTAS * kSortThreads) * kSortThreads) : 0;
  const auto bytes = [](int digit, int room) {
    return static_cast<size_t>(kSortWarps + CTAS + 1) * (size_t(1) << digit) * sizeof(int) +
           static_cast<size_t>(room) * sizeof(uint64_t);
  };
  static std::atomic<int> configured[64];  // (several threads may come here at once)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(token_sort_kernel<CTAS, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes(kSortDigit, SHARED ? kSortRoom : 0)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(1, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CTAS);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = bytes(p.digit, p.room);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CTAS;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CTAS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, token_sort_kernel<CTAS, SHARED>, p);
}

cudaError_t sort_tokens(SortParams p, cudaStream_t s) {
  int bits = 1;
  while ((int64_t(1) << bits) <= p.V) ++bits;  // keys go up to V
  p.passes = (bits + kSortDigit - 1) / kSortDigit;
  p.digit = (bits + p.passes - 1) / p.passes;
  prof_begin(s, FLCE_KERNEL_TOKEN_SORT);
  const cudaError_t e = p.N <= kSortAlone              ? launch_sort<1, true>(p, s)
                        : p.N <= kSortRoom * kSortCtas ? launch_sort<kSortCtas, true>(p, s)
                                                       : launch_sort<kSortCtas, false>(p, s);
  prof_end(s);
  return e;
}

// Pieces of a row of H columns, each a warp's.
template <typename T>
int64_t row_pieces(int64_t H, bool vectors) {
  return div_up(H, vectors ? 32 * (16 / static_cast<int64_t>(sizeof(T))) : 32 * 4);
}

template <typename T>
cudaError_t sum_rows(SumParams p, bool vectors, bool few, cudaStream_t s) {
  constexpr int kE = 16 / sizeof(T);
  p.columns = static_cast<int>(row_pieces<T>(p.H, vectors));
  cudaError_t e;
  prof_begin(s, FLCE_KERNEL_EMBEDDING_BWD);
  if (few) {
    p.zero_ctas = p.accumulate ? 0 : static_cast<unsigned>(div_up(p.V, kFewZeroRows) * div_up(p.H, kFewZeroColumns));
    const unsigned grid = static_cast<unsigned>(p.N) * p.columns + p.zero_ctas;
    if (vectors)
      embedding_few_kernel<T, kE, 1><<<grid, 32 * kFewWarps, 0, s>>>(p);
    else
      embedding_few_kernel<T, 1, 4><<<grid, 32 * kFewWarps, 0, s>>>(p);
    e = cudaGetLastError();
  } else {
    p.zero_ctas = p.accumulate ? 0 : static_cast<unsigned>(std::min<int64_t>(8 * device_sm_count(), div_up(p.V, kSumWarps)));
    const dim3 grid(static_cast<unsigned>(p.zero_ctas + div_up(static_cast<int64_t>(p.tiles) * p.columns, kSumWarps)));
    constexpr size_t kRingBytes = sizeof(uint4) * kSumWarps * kRing * 32;
    e = vectors ? launch_after_with(kRingBytes, embedding_sum_kernel<T, kE, 1>, grid, dim3(32 * kSumWarps), s, p)
                : launch_after(embedding_sum_kernel<T, 1, 4>, grid, dim3(32 * kSumWarps), s, p);
  }
  prof_end(s);
  return e;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

flce_status_t embedding_fwd(int dtype, const void* table, int64_t ld_table, const void* ids, int index_type, int64_t N,
                            int64_t V, int64_t H, float scale, void* y, int64_t ld_y, int32_t* status_dev,
                            flce_stream_t stream_) {
  if (!float_dtype(dtype)) return FLCE_ERR_UNSUPPORTED;
  if (index_type != FLCE_INDEX_INT64 && index_type != FLCE_INDEX_INT32) return FLCE_ERR_INVALID_ARG;
  const int64_t most = int64_t(1) << 31, far = int64_t(1) << 58;
  if (N < 0 || N >= most || V < 1 || V >= most || H < 1 || H >= (1 << 24)) return FLCE_ERR_INVALID_ARG;
  if (ld_table < H || ld_table > far / V || ld_y < H || ld_y > far / (N > 0 ? N : 1)) return FLCE_ERR_INVALID_ARG;
  if (table == nullptr || (N > 0 && (ids == nullptr || y == nullptr))) return FLCE_ERR_INVALID_ARG;
  const size_t esz = elem_size(dtype);
  if (!aligned_to(table, esz) || !aligned_to(y, esz) || !aligned_to(ids, index_type == FLCE_INDEX_INT64 ? 8 : 4) ||
      !aligned_to(status_dev, 4))
    return FLCE_ERR_MISALIGNED;
  if (N == 0) return FLCE_OK;
  const uintptr_t a = reinterpret_cast<uintptr_t>(table), b = reinterpret_cast<uintptr_t>(y);
  if (a < b + ((N - 1) * ld_y + H) * esz && b < a + ((V - 1) * ld_table + H) * esz) return FLCE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  const LookupParams p = {table, ids, y, ld_table, ld_y, N, V, H, 0, index_type == FLCE_INDEX_INT32, scale, status_dev};
  const cudaError_t e = dtype == FLCE_DTYPE_BF16   ? lookup<__nv_bfloat16>(p, s)
                        : dtype == FLCE_DTYPE_FP16 ? lookup<__half>(p, s)
                                                   : lookup<float>(p, s);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

size_t embedding_workspace_size(int64_t N, int64_t V, int64_t H) {
  EmbeddingLayout at;
  return embedding_layout(N, V, H, &at) && launches_hold(N, H) ? at.total : 0;
}

flce_status_t embedding_bwd(int dtype, const void* grad_y, int64_t ld_grad_y, const void* ids, int index_type,
                            int64_t N, int64_t V, int64_t H, float scale, int64_t padding_index, float* grad_table,
                            int accumulate, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                            flce_stream_t stream_) {
  EmbeddingLayout at;
  if (!float_dtype(dtype)) return FLCE_ERR_UNSUPPORTED;
  if (index_type != FLCE_INDEX_INT64 && index_type != FLCE_INDEX_INT32) return FLCE_ERR_INVALID_ARG;
  if (!embedding_layout(N, V, H, &at) || (accumulate != 0 && accumulate != 1)) return FLCE_ERR_INVALID_ARG;
  if (ld_grad_y < 0 || ld_grad_y > (int64_t(1) << 58) / (N > 0 ? N : 1)) return FLCE_ERR_INVALID_ARG;
  if (padding_index < -1 || padding_index >= V) return FLCE_ERR_INVALID_ARG;
  if (grad_table == nullptr || (N > 0 && (grad_y == nullptr || ids == nullptr))) return FLCE_ERR_INVALID_ARG;
  const size_t esz = elem_size(dtype);
  if (!aligned_to(grad_y, esz) || !aligned_to(grad_table, 4) || !aligned_to(status_dev, 4) ||
      !aligned_to(ids, index_type == FLCE_INDEX_INT64 ? 8 : 4))
    return FLCE_ERR_MISALIGNED;
  if (N > 0) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(grad_y), b = reinterpret_cast<uintptr_t>(grad_table);
    if (a < b + static_cast<uintptr_t>(V) * H * 4 && b < a + ((N - 1) * ld_grad_y + H) * esz)
      return FLCE_ERR_INVALID_ARG;
  }
  if (!launches_hold(N, H)) return FLCE_ERR_UNSUPPORTED;
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < at.total) return FLCE_ERR_WORKSPACE;
  if (N == 0 && accumulate) return FLCE_OK;
  const int64_t tiles = div_up(N, kTile);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  // without the sort (11 us) where the CTAs that compare ids are few
  const bool vectors = aligned_to(grad_y, 16) && aligned_to(grad_table, 16) && H % (16 / esz) == 0 &&
                          (ld_grad_y % static_cast<int64_t>(16 / esz) == 0 || N <= 1);
  const bool few = N <= kFewTokens && N * div_up(H, vectors ? 32 * (16 / esz) : 128) <= kFewCtas &&
                   div_up(V, kFewZeroRows) * div_up(H, kFewZeroColumns) < (int64_t(1) << 30);
  SortParams sort = {};
  sort.ids = ids, sort.ids32 = index_type == FLCE_INDEX_INT32;
  sort.N = static_cast<int>(N), sort.V = static_cast<int>(V), sort.padding = padding_index;
  for (int k = 0; k < 2; ++k) {
    sort.keys[k] = reinterpret_cast<int*>(ws + at.keys[k]);
    sort.tokens[k] = reinterpret_cast<int*>(ws + at.tokens[k]);
  }
  sort.hit = accumulate ? nullptr : reinterpret_cast<uint32_t*>(ws + at.hit);
  sort.status = status_dev;
  if (!few && sort_tokens(sort, s) != cudaSuccess) return FLCE_ERR_CUDA;

  SumParams p = {};
  p.grad_y = grad_y, p.ld = ld_grad_y, p.H = H, p.N = sort.N, p.V = sort.V;
  p.keys = sort.keys[0], p.tokens = sort.tokens[0], p.hit = sort.hit;
  p.table = grad_table, p.partial = reinterpret_cast<float*>(ws + at.partial);
  p.joins = reinterpret_cast<int*>(ws + at.joins);
  p.accumulate = accumulate, p.scale = scale, p.tiles = static_cast<int>(tiles);
  p.ids = ids, p.ids32 = sort.ids32, p.padding = padding_index, p.status = status_dev;
  const cudaError_t e = dtype == FLCE_DTYPE_BF16   ? sum_rows<__nv_bfloat16>(p, vectors, few, s)
                        : dtype == FLCE_DTYPE_FP16 ? sum_rows<__half>(p, vectors, few, s)
                                                   : sum_rows<float>(p, vectors, few, s);
  if (e != cudaSuccess) return FLCE_ERR_CUDA;
  if (!few) {
    const unsigned columns = static_cast<unsigned>(div_up(H, vectors ? 128 : 32));
    prof_begin(s, FLCE_KERNEL_EMBEDDING_JOIN);
    const int64_t most = std::max<int64_t>(1, 4096 / columns);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(div_up(tiles, kJoinTiles), most)), columns);
    const cudaError_t j = launch_after(vectors ? embedding_join_kernel<4> : embedding_join_kernel<1>, grid,
                                       dim3(32 * kJoinWarps), s, p);
    prof_end(s);
    if (j != cudaSuccess) return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}

}  // extern "C"
