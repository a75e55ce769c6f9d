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

// A part of a row by each warp.
template <typename T, int E>
__global__ void __launch_bounds__(32 * kLookupWarps) embedding_kernel(const LookupParams p) {
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
      *reinterpret_cast<Elems<T, E>*>(to + at) = v[i];
    }
  }
}

template <typename T>
cudaError_t lookup(LookupParams p, cudaStream_t s) {
  constexpr int kE = 16 / sizeof(T);
  const bool vectors = aligned_to(p.table, 16) && aligned_to(p.y, 16) && p.H % kE == 0 &&
                       (p.ld_table % kE == 0 || p.V == 1) && (p.ld_y % kE == 0 || p.N == 1);
  p.parts = div_up(p.H, 32 * kLookupUnroll * (vectors ? kE : 1));
  const int64_t ctas = div_up(p.N * p.parts, kLookupWarps), most = int64_t(1) << 30;
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  prof_begin(s, FLCE_KERNEL_EMBEDDING);
  if (vectors)
    embedding_kernel<T, kE><<<grid, 32 * kLookupWarps, 0, s>>>(p);
  else
    embedding_kernel<T, 1><<<grid, 32 * kLookupWarps, 0, s>>>(p);
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
  int* keys[2];        // [N] each; the result is in keys[0], tokens[0]
  int* tokens[2];
  uint32_t* hit;       // a bit for each row of the table that gets something, or null
  int* status;
};

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortDigit = 9;  // most bits of a pass: two passes reach 2^18 ids

// Stable radix sort, least significant digit first, by one cluster.  Each warp owns a
// stretch of the list: it counts its digits, the counts are added up over warps and CTAs
// (through distributed shared memory), and it puts its keys where those before them leave
// room.  Lanes with the same digit find one another by match.
__global__ void __launch_bounds__(kSortThreads) token_sort_kernel(const SortParams p) {
  extern __shared__ int counts[];  // [warps][digits], then [digits] of the CTA, then scratch of the scan
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << p.digit;
  int* own = counts + warp * digits;
  int* totals = counts + kSortWarps * digits;
  __shared__ int warp_sums[32];
  const unsigned rank = cluster_cta_rank();
  unsigned ctas;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const int64_t warps = static_cast<int64_t>(ctas) * kSortWarps;
  const int64_t stretch = (p.N + warps * 32 - 1) / (warps * 32) * 32;
  const int64_t from = (static_cast<int64_t>(rank) * kSortWarps + warp) * stretch;
  const int64_t to = from + stretch < p.N ? from + stretch : p.N;
  if (p.hit != nullptr) {
    for (int i = rank * kSortThreads + threadIdx.x; i < (p.V + 31) / 32; i += ctas * kSortThreads) p.hit[i] = 0;
    cluster_sync_all();
  }
  int bits = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    // the last pass ends in array 0; pass 0 reads the ids themselves
    const int to_array = (p.passes - 1 - pass) & 1;
    const int* keys = p.keys[to_array ^ 1];
    const int* tokens = p.tokens[to_array ^ 1];
    const int shift = pass * p.digit;
    const auto key_of = [&](int64_t i) -> int {
      if (pass > 0) return __ldcg(keys + i);
      const int64_t id = id_at(p.ids, p.ids32, i);
      return id < 0 || id >= p.V || id == p.padding ? p.V : static_cast<int>(id);
    };
    for (int d = lane; d < digits; d += 32) own[d] = 0;
    __syncwarp();
    for (int64_t i0 = from; i0 < to; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool valid = i < to;
      const int key = valid ? key_of(i) : 0;
      if (pass == 0 && valid) {
        const int64_t id = id_at(p.ids, p.ids32, i);
        if (id < 0 || id >= p.V) bits |= FLCE_STATUS_BIT_TARGET_RANGE;
        // (frequent ids would queue up at their word)
        if (p.hit != nullptr && key < p.V && !(__ldcg(p.hit + (key >> 5)) >> (key & 31) & 1))
          atomicOr(p.hit + (key >> 5), 1u << (key & 31));
      }
      const int d = valid ? (key >> shift) & (digits - 1) : -1;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (valid && lane == __ffs(same) - 1) own[d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // counts of the CTA's warps become those before each, and the CTA's totals
    for (int d = threadIdx.x; d < digits; d += kSortThreads) {
      int sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = counts[w * digits + d];
        counts[w * digits + d] = sum;
        sum += c;
      }
      totals[d] = sum;
    }
    cluster_sync_all();
    // where a digit's keys start: after all smaller digits, and those of the CTAs before
    int before = 0, all = 0;
    const int d = threadIdx.x;  // digits <= threads
    if (d < digits) {
      for (unsigned r = 0; r < ctas; ++r) {
        int c;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(map_to_cta(smem_addr(totals + d), r)) : "memory");
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
    int start = scan - all + before;
    for (int w = 0; w < warp; ++w) start += warp_sums[w];
    if (d < digits)
      for (int w = 0; w < kSortWarps; ++w) counts[w * digits + d] += start;
    __syncthreads();
    for (int64_t i0 = from; i0 < to; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool valid = i < to;
      const int key = valid ? key_of(i) : 0;
      const int digit = valid ? (key >> shift) & (digits - 1) : -1;
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      int at = 0;
      if (valid) at = own[digit] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (valid && lane == __ffs(same) - 1) own[digit] += __popc(same);
      if (valid) {
        p.keys[to_array][at] = key;
        p.tokens[to_array][at] = pass > 0 ? __ldcg(tokens + i) : static_cast<int>(i);
      }
      __syncwarp();
    }
    cluster_sync_all();  // every CTA's keys are in place, and its totals have been read
  }
  if (bits != 0 && p.status != nullptr) atomicOr(p.status, bits);
}

// ---------------------------------------------------------------- sums

constexpr int kTile = 32;          // sorted tokens of a tile
constexpr int kSumThreads = 128;

struct SumParams {
  const void* grad_y;
  int64_t ld, H;
  int N, V;
  const int* keys;
  const int* tokens;
  const uint32_t* hit;  // null: rows without tokens are not written
  float* table;
  float* partial;       // [tiles][2][H]: what a tile has of an id that began before it, and of one that goes on
  int accumulate;
  float scale;
  int tiles, columns;   // the grid's tiles, and its pieces of a row
};

// One tile's columns by each CTA; the CTAs after those write zeros to the table's rows that
// get nothing.  A thread has GROUPS times E columns and goes through the tile's tokens in
// order.
template <typename T, int E, int GROUPS>
__global__ void __launch_bounds__(kSumThreads) embedding_sum_kernel(const SumParams p) {
  constexpr int kAhead = 8 / GROUPS < 1 ? 1 : 8 / GROUPS;  // tokens that are loaded at a time
  __shared__ int keys[kTile + 2], tokens[kTile];
  grid_dependency_wait();
  if (blockIdx.x >= static_cast<unsigned>(p.tiles) * p.columns) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = (blockIdx.x - p.tiles * p.columns) * (kSumThreads / 32) + warp;
    const int step = (gridDim.x - p.tiles * p.columns) * (kSumThreads / 32);
    for (int64_t v = first; v < p.V; v += step) {
      if (__ldg(p.hit + (v >> 5)) >> (v & 31) & 1) continue;
      float* row = p.table + v * p.H;
      if constexpr (E > 1) {
        for (int64_t h = lane * 4; h < p.H; h += 128) __stcs(reinterpret_cast<float4*>(row + h), make_float4(0, 0, 0, 0));
      } else {
        for (int64_t h = lane; h < p.H; h += 32) __stcs(row + h, 0.f);
      }
    }
    return;
  }
  const int tile = blockIdx.x / p.columns, column = blockIdx.x % p.columns;
  const int64_t begin = static_cast<int64_t>(tile) * kTile;
  const int count = static_cast<int>(p.N - begin < kTile ? p.N - begin : kTile);
  // keys[0] and keys[count + 1] are the neighbours' (-1 beyond the list)
  for (int i = threadIdx.x; i < count + 2; i += kSumThreads) {
    const int64_t at = begin + i - 1;
    keys[i] = at >= 0 && at < p.N ? p.keys[at] : -1;
  }
  for (int i = threadIdx.x; i < count; i += kSumThreads) tokens[i] = p.tokens[begin + i];
  __syncthreads();
  const int64_t first = (static_cast<int64_t>(column) * GROUPS * kSumThreads + threadIdx.x) * E;
  float sum[GROUPS][E];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g)
#pragma unroll
    for (int k = 0; k < E; ++k) sum[g][k] = 0.f;
  int start = 0;  // where the present id's tokens start
  for (int t0 = 0; t0 < count; t0 += kAhead) {
    Elems<T, E> v[kAhead][GROUPS];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (t0 + a < count && keys[t0 + a + 1] < p.V) {
        const T* row = static_cast<const T*>(p.grad_y) + tokens[t0 + a] * p.ld;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const int64_t h = first + static_cast<int64_t>(g) * kSumThreads * E;
          if (h < p.H) v[a][g] = *reinterpret_cast<const Elems<T, E>*>(row + h);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int t = t0 + a;
      if (t >= count) break;
      const int key = keys[t + 1];
      if (key >= p.V) break;  // tokens that add nothing end the list
#pragma unroll
      for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int k = 0; k < E; ++k) sum[g][k] += to_float(v[a][g].v[k]);
      if (t + 1 < count && keys[t + 2] == key) continue;
      // the id's last token in this tile
      const bool began_before = start == 0 && keys[0] == key, goes_on = keys[t + 2] == key;
      float* to;
      if (began_before || goes_on)
        to = p.partial + (static_cast<int64_t>(tile) * 2 + (began_before ? 0 : 1)) * p.H;
      else
        to = p.table + key * p.H;
      const bool whole = !began_before && !goes_on;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const int64_t h = first + static_cast<int64_t>(g) * kSumThreads * E;
        if (h < p.H) {
          if constexpr (E > 1) {
#pragma unroll
            for (int q = 0; q < E; q += 4) {
              float4* at = reinterpret_cast<float4*>(to + h + q);
              float4 o = make_float4(sum[g][q], sum[g][q + 1], sum[g][q + 2], sum[g][q + 3]);
              if (whole) {
                o = make_float4(o.x * p.scale, o.y * p.scale, o.z * p.scale, o.w * p.scale);
                if (p.accumulate) {
                  const float4 old = *at;
                  o = make_float4(old.x + o.x, old.y + o.y, old.z + o.z, old.w + o.w);
                }
              }
              *at = o;
            }
          } else {
            float o = sum[g][0];
            if (whole) {
              o *= p.scale;
              if (p.accumulate) o += to[h];
            }
            to[h] = o;
          }
        }
#pragma unroll
        for (int k = 0; k < E; ++k) sum[g][k] = 0.f;
      }
      start = t + 1;
    }
  }
}

constexpr int kJoinWarps = 8;

// Adds up the partial rows of an id that goes over several tiles, in the order of the
// tiles: each warp a stretch of them, then the warps' sums.  A CTA has 32 * E columns and
// looks at tiles for such ids that begin there.
template <int E>
__global__ void __launch_bounds__(32 * kJoinWarps) embedding_join_kernel(const SumParams p) {
  using V = Elems<float, E>;
  __shared__ V sums[kJoinWarps][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t h = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * E;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int64_t begin = static_cast<int64_t>(tile) * kTile, end = begin + kTile;
    if (end >= p.N) return;
    const int key = __ldg(p.keys + end - 1);
    if (key >= p.V || __ldg(p.keys + end) != key) continue;  // nothing goes on
    if (begin > 0 && __ldg(p.keys + begin) == key && __ldg(p.keys + begin - 1) == key) continue;  // it began before
    // the id's last token, by bisection: keys[low] == key
    int64_t low = end, high = p.N;
    while (high - low > 1) {
      const int64_t mid = low + (high - low) / 2;
      if (__ldg(p.keys + mid) == key)
        low = mid;
      else
        high = mid;
    }
    const int parts = static_cast<int>(low / kTile) - tile + 1;
    const int each = (parts + kJoinWarps - 1) / kJoinWarps;
    V sum = {};
    if (h < p.H) {
      const int to = (warp + 1) * each < parts ? (warp + 1) * each : parts;
#pragma unroll 8
      for (int i = warp * each; i < to; ++i) {
        const V v = *reinterpret_cast<const V*>(p.partial + (static_cast<int64_t>(tile + i) * 2 + (i == 0)) * p.H + h);
#pragma unroll
        for (int k = 0; k < E; ++k) sum.v[k] += v.v[k];
      }
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && h < p.H) {
      V* at = reinterpret_cast<V*>(p.table + key * p.H + h);
      V out = {};
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

struct EmbeddingLayout {
  size_t keys[2], tokens[2], hit, partial, total;
};

bool embedding_layout(int64_t N, int64_t V, int64_t H, EmbeddingLayout* at) {
  if (N < 0 || N >= (int64_t(1) << 31) - kTile || V < 1 || V >= (int64_t(1) << 31) - 1 || H < 1 || H >= (1 << 24))
    return false;
  const size_t list = align_up(static_cast<size_t>(N) * 4, 256);
  at->keys[0] = 0, at->keys[1] = list, at->tokens[0] = 2 * list, at->tokens[1] = 3 * list;
  at->hit = 4 * list;
  at->partial = align_up(at->hit + static_cast<size_t>(div_up(V, 32)) * 4, 256);
  at->total = align_up(at->partial + static_cast<size_t>(div_up(N, kTile)) * 2 * H * 4, 256);
  return true;
}

cudaError_t sort_tokens(SortParams p, cudaStream_t s) {
  int bits = 1;
  while ((int64_t(1) << bits) <= p.V) ++bits;  // keys go up to V
  p.passes = (bits + kSortDigit - 1) / kSortDigit;
  p.digit = (bits + p.passes - 1) / p.passes;
  const size_t smem = (static_cast<size_t>(kSortWarps) + 1) * (size_t(1) << p.digit) * sizeof(int);
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(token_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (kSortWarps + 1) * (1 << kSortDigit) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const int ctas = p.N <= 4096 ? 1 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_begin(s, FLCE_KERNEL_TOKEN_SORT);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, token_sort_kernel, p);
  prof_end(s);
  return e;
}

template <typename T>
cudaError_t sum_rows(SumParams p, bool vectors, cudaStream_t s) {
  constexpr int kE = 16 / sizeof(T);
  p.columns = static_cast<int>(div_up(p.H, vectors ? kSumThreads * kE : kSumThreads * 4));
  const int64_t ctas = static_cast<int64_t>(p.tiles) * p.columns + (p.hit != nullptr ? 8 * device_sm_count() : 0);
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  if (ctas == 0) return cudaSuccess;
  prof_begin(s, FLCE_KERNEL_EMBEDDING_BWD);
  const dim3 grid(static_cast<unsigned>(ctas));
  const cudaError_t e = vectors ? launch_after(embedding_sum_kernel<T, kE, 1>, grid, dim3(kSumThreads), s, p)
                                : launch_after(embedding_sum_kernel<T, 1, 4>, grid, dim3(kSumThreads), s, p);
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
  return embedding_layout(N, V, H, &at) ? at.total : 0;
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
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < at.total) return FLCE_ERR_WORKSPACE;
  if (N == 0 && accumulate) return FLCE_OK;
  const int64_t tiles = div_up(N, kTile);
  if (tiles * div_up(H, kSumThreads * 4) + 8 * 1024 >= (int64_t(1) << 31) || div_up(H, 32) > 65535)
    return FLCE_ERR_UNSUPPORTED;  // more CTAs than a launch has
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  SortParams sort = {};
  sort.ids = ids, sort.ids32 = index_type == FLCE_INDEX_INT32;
  sort.N = static_cast<int>(N), sort.V = static_cast<int>(V), sort.padding = padding_index;
  for (int k = 0; k < 2; ++k) {
    sort.keys[k] = reinterpret_cast<int*>(ws + at.keys[k]);
    sort.tokens[k] = reinterpret_cast<int*>(ws + at.tokens[k]);
  }
  sort.hit = accumulate ? nullptr : reinterpret_cast<uint32_t*>(ws + at.hit);
  sort.status = status_dev;
  if (sort_tokens(sort, s) != cudaSuccess) return FLCE_ERR_CUDA;

  SumParams p = {};
  p.grad_y = grad_y, p.ld = ld_grad_y, p.H = H, p.N = sort.N, p.V = sort.V;
  p.keys = sort.keys[0], p.tokens = sort.tokens[0], p.hit = sort.hit;
  p.table = grad_table, p.partial = reinterpret_cast<float*>(ws + at.partial);
  p.accumulate = accumulate, p.scale = scale, p.tiles = static_cast<int>(tiles);
  const int64_t elems = 16 / static_cast<int64_t>(esz);
  const bool vectors =
      aligned_to(grad_y, 16) && aligned_to(grad_table, 16) && H % elems == 0 && (ld_grad_y % elems == 0 || N == 1);
  const cudaError_t e = dtype == FLCE_DTYPE_BF16   ? sum_rows<__nv_bfloat16>(p, vectors, s)
                        : dtype == FLCE_DTYPE_FP16 ? sum_rows<__half>(p, vectors, s)
                                                   : sum_rows<float>(p, vectors, s);
  if (e != cudaSuccess) return FLCE_ERR_CUDA;
  if (tiles > 1) {
    const unsigned columns = static_cast<unsigned>(div_up(H, vectors ? 128 : 32));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tiles, std::max<int64_t>(2048 / columns, 1))), columns);
    prof_begin(s, FLCE_KERNEL_EMBEDDING_JOIN);
    const cudaError_t j = launch_after(vectors ? embedding_join_kernel<4> : embedding_join_kernel<1>, grid,
                                       dim3(32 * kJoinWarps), s, p);
    prof_end(s);
    if (j != cudaSuccess) return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}

}  // extern "C"
