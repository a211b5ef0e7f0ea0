// expert_sort_kernel.cu -- the order by expert of n = tokens * k expert ids:
//
//   offsets[e]  = number of entries with a valid id below e,
//   position[i] = offsets[id_i] + number of entries before i with the same id,
//
// a stable counting sort (-1 for an id outside [0, experts)). The entries are cut into chunks, a
// CTA each, and a chunk into one run of neighbours a warp, ITEMS a lane in registers. One kernel
// counts every chunk's ids; the next ranks its own entries 32 at a time -- lanes with one id find
// each other by a warp match, and the warp's running count of that id gives their places in its
// run -- and meanwhile adds up the counts of the chunks before its own and of the experts before
// each (every CTA for itself, from L2: at most 128 chunks until a lane's entries no longer fit its
// registers), then of its warps. All counts are integers: the same ids give the same order. Up to
// 2048 entries take one launch.
//
// Bound by latency, a chain of loads, matches, prefix sums and stores (one GB300: 256 entries
// 2.9 us, 65536 6.6, calls one after another).
#include <algorithm>

#include "expert_internal.h"
#include "pdl.h"
#include "ptx.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kMaxChunks = 128;  // of up to 16 entries a thread

struct SortParams {
  const void *ids;
  int64_t ld_ids;
  int64_t n;
  int32_t k, experts, chunk, chunks;
  int32_t wide, flat;  // 8-byte ids; rows of ids follow one another
  int32_t *position, *offsets;
  int32_t *counts;  // [chunks][experts]
};

// Expert of entry i, or -1.
__device__ __forceinline__ int id_at(const SortParams &p, int64_t i) {
  int64_t at = i;
  if (!p.flat) {
    const uint32_t t = static_cast<uint32_t>(i) / static_cast<uint32_t>(p.k);
    at = t * p.ld_ids + (static_cast<uint32_t>(i) - t * static_cast<uint32_t>(p.k));
  }
  const int64_t id = p.wide ? static_cast<const int64_t *>(p.ids)[at]
                            : static_cast<int64_t>(static_cast<const int32_t *>(p.ids)[at]);
  return id >= 0 && id < p.experts ? static_cast<int>(id) : -1;
}

__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const SortParams p) {
  extern __shared__ int32_t count[];  // [experts]
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int64_t hi = min(lo + p.chunk, p.n);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
    const int id = id_at(p, i);
    if (id >= 0) atomicAdd(&count[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads)
    p.counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] = count[e];
}

template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const SortParams p) {
  extern __shared__ int32_t smem[];
  const int E = p.experts;
  int32_t *total = smem;            // [E]: entries of each expert, then their first rows
  int32_t *before = total + E;      // [E]: those in earlier chunks
  int32_t *cursor = before + E;     // [warps][E]
  int32_t *warp_sum = cursor + kSortWarps * E;  // [warps]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int i = threadIdx.x; i < (2 + kSortWarps) * E; i += kSortThreads) smem[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  // This warp's run of the chunk: every lane's entries, and their places among the run's entries
  // of the same expert.
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.chunk + warp * (32 * ITEMS);
  int id[ITEMS], place[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t at = lo + i * 32 + lane;
    id[i] = at < p.n ? id_at(p, at) : -1;
  }
  int32_t *mine = cursor + warp * E;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (lo + i * 32 >= p.n) break;
    const unsigned same = __match_any_sync(0xffffffffu, id[i]);
    const int rank = __popc(same & ((1u << lane) - 1));
    const int at = id[i] >= 0 ? mine[id[i]] : 0;
    __syncwarp();  // every lane has read its count
    if (id[i] >= 0 && rank == 0) mine[id[i]] = at + __popc(same);
    __syncwarp();
    place[i] = at + rank;
  }
  if (p.chunks > 1) {
    // groups of threads take every so many-th chunk, a thread one expert
    const int width = (E + 31) / 32 * 32, groups = max(1, kSortThreads / width);
    const int g = static_cast<int>(threadIdx.x) / width;
    if (g < groups)
      for (int e = static_cast<int>(threadIdx.x) - g * width; e < E; e += kSortThreads) {
        int all = 0, earlier = 0;
#pragma unroll 8
        for (int c = g; c < p.chunks; c += groups) {
          const int v = p.counts[static_cast<int64_t>(c) * E + e];
          all += v;
          earlier += c < static_cast<int>(blockIdx.x) ? v : 0;
        }
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], earlier);
      }
  }
  __syncthreads();
  if (p.chunks == 1) {
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
      int t = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) t += cursor[w * E + e];
      total[e] = t;
    }
    __syncthreads();
  }
  // Exclusive prefix sums over the experts: two a thread (at most 1024).
  const int e0 = 2 * static_cast<int>(threadIdx.x), e1 = e0 + 1;
  const int t0 = e0 < E ? total[e0] : 0, t1 = e1 < E ? total[e1] : 0;
  int sum = t0 + t1;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += v;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int first = sum - t0 - t1;
  for (int w = 0; w < warp; ++w) first += warp_sum[w];
  if (e0 < E) total[e0] = first;
  if (e1 < E) total[e1] = first + t0;
  if (blockIdx.x == 0) {
    if (e0 < E) p.offsets[e0] = first;
    if (e1 < E) p.offsets[e1] = first + t0;
    if (threadIdx.x == 0) {
      int all = 0;
      for (int w = 0; w < kSortWarps; ++w) all += warp_sum[w];
      p.offsets[E] = all;
    }
  }
  __syncthreads();
  // Every warp's first position of each expert.
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int at = total[e] + before[e];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = cursor[w * E + e];
      cursor[w * E + e] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t at = lo + i * 32 + lane;
    if (at < p.n) p.position[at] = id[i] >= 0 ? mine[id[i]] + place[i] : -1;
  }
}

// Entries a lane holds: 4, 8 or 16, and 16 for any longer list.
int items_of(int64_t n) {
  int items = 4;
  while (items < 16 && n > kMaxChunks * kSortThreads * items) items *= 2;
  return items;
}

// All of expert_place_kernel's shared memory (none is static: 48 KB is the limit of both together).
constexpr size_t place_bytes(int64_t experts) {
  return static_cast<size_t>((2 + kSortWarps) * experts + kSortWarps) * sizeof(int32_t);
}

template <int ITEMS>
cudaError_t place_launch(const SortParams &p, dim3 grid, size_t smem, cudaStream_t s) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        expert_place_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(place_bytes(kMaxExperts)));
    if (e != cudaSuccess) return e;
  }
  launch_pdl(expert_place_kernel<ITEMS>, grid, kSortThreads, smem, s, p);
  return cudaGetLastError();
}

}  // namespace

size_t expert_sort_bytes(int64_t n, int64_t experts) {
  const int64_t chunk = static_cast<int64_t>(kSortThreads) * items_of(n), chunks = (n + chunk - 1) / chunk;
  return chunks > 1 ? static_cast<size_t>(chunks * experts) * sizeof(int32_t) : 0;
}

cudaError_t expert_sort_launch(const void *ids, int64_t ld_ids, bool wide, int64_t tokens, int64_t k,
                               int64_t experts, int32_t *position, int32_t *offsets,
                               void *workspace, int *launches, cudaStream_t s) {
  SortParams p{};
  p.ids = ids, p.ld_ids = ld_ids, p.wide = wide;
  p.flat = tokens <= 1 || ld_ids == k;
  p.n = tokens * k;
  p.k = static_cast<int32_t>(std::max<int64_t>(k, 1));
  p.experts = static_cast<int32_t>(experts);
  const int items = items_of(p.n);
  const int64_t chunk = static_cast<int64_t>(kSortThreads) * items;
  const int64_t chunks = std::max<int64_t>((p.n + chunk - 1) / chunk, 1);
  p.chunk = static_cast<int32_t>(chunk), p.chunks = static_cast<int32_t>(chunks);
  p.position = position, p.offsets = offsets;
  p.counts = static_cast<int32_t *>(workspace);
  const dim3 grid(static_cast<unsigned>(chunks));
  *launches = chunks > 1 ? 2 : 1;
  if (chunks > 1) launch_pdl(expert_count_kernel, grid, kSortThreads, experts * sizeof(int32_t), s, p);
  const size_t smem = place_bytes(experts);
  switch (items) {
    case 4: return place_launch<4>(p, grid, smem, s);
    case 8: return place_launch<8>(p, grid, smem, s);
    default: return place_launch<16>(p, grid, smem, s);
  }
}

}  // namespace ff
}  // namespace gemm_gb300
