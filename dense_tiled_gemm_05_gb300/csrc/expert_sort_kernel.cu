// expert_sort_kernel.cu -- the order by expert of n = tokens * k expert ids:
//
//   offsets[e]  = number of entries with a valid id below e,
//   position[i] = offsets[id_i] + number of entries before i with the same id,
//
// a stable counting sort (-1 for an id outside [0, experts)). The entries are cut into chunks, a
// CTA each, and a chunk into one run of neighbours a warp. One kernel counts every chunk's ids;
// the next adds up the counts of the chunks before its own and of the experts before each (every
// CTA for itself: at most 128 chunks, so up to half a megabyte from L2), then of its own warps
// before each, and gives out positions 32 entries at a time: lanes with one id find each other
// by a warp match and are ranked by lane. All counts are integers: the same ids give the same
// order. Up to kChunk entries take one launch.
//
// Bound by latency: a chain of loads, counts, prefix sums and stores.
#include <algorithm>

#include "expert_internal.h"
#include "pdl.h"
#include "ptx.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kChunk = 2048;     // least entries a CTA
constexpr int64_t kMaxChunks = 128;

struct SortParams {
  const void *ids;
  int64_t ld_ids;
  int64_t n;
  int32_t k, experts, chunk, chunks;
  int32_t wide;
  int32_t *position, *offsets;
  int32_t *counts;  // [chunks][experts]
};

// Expert of entry i, or -1.
__device__ __forceinline__ int id_at(const SortParams &p, int64_t i) {
  const int64_t t = i / p.k, at = t * p.ld_ids + (i - t * p.k);
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

__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const SortParams p) {
  extern __shared__ int32_t smem[];
  const int E = p.experts;
  int32_t *total = smem;            // [E]: entries of each expert, then their first rows
  int32_t *before = total + E;      // [E]: those in earlier chunks
  int32_t *cursor = before + E;     // [warps][E]
  __shared__ int32_t warp_sum[kSortWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int i = threadIdx.x; i < (2 + kSortWarps) * E; i += kSortThreads) smem[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  // This warp's run of the chunk.
  const int64_t run = (p.chunk + kSortWarps - 1) / kSortWarps;
  const int64_t end = min(static_cast<int64_t>(blockIdx.x + 1) * p.chunk, p.n);
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.chunk + warp * run;
  const int64_t hi = min(lo + run, end);
  int32_t *mine = cursor + warp * E;
  for (int64_t i = lo + lane; i < hi; i += 32) {
    const int id = id_at(p, i);
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  if (p.chunks > 1) {
    for (int c = warp; c < p.chunks; c += kSortWarps)
      for (int e = lane; e < E; e += 32) {
        const int v = p.counts[static_cast<int64_t>(c) * E + e];
        if (v) atomicAdd(&total[e], v);
        if (v && c < static_cast<int>(blockIdx.x)) atomicAdd(&before[e], v);
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
  for (int64_t i0 = lo; i0 < hi; i0 += 32) {
    const int64_t i = i0 + lane;
    const int id = i < hi ? id_at(p, i) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1));
    const int at = id >= 0 ? mine[id] : 0;
    __syncwarp();  // every lane has read its cursor
    if (id >= 0 && rank == 0) mine[id] = at + __popc(same);
    __syncwarp();
    if (i < hi) p.position[i] = id >= 0 ? at + rank : -1;
  }
}

int64_t chunk_of(int64_t n) {
  const int64_t even = (n + kMaxChunks - 1) / kMaxChunks;
  return even > kChunk ? (even + 511) / 512 * 512 : kChunk;
}

}  // namespace

size_t expert_sort_bytes(int64_t n, int64_t experts) {
  const int64_t chunk = chunk_of(n), chunks = (n + chunk - 1) / chunk;
  return chunks > 1 ? static_cast<size_t>(chunks * experts) * sizeof(int32_t) : 0;
}

cudaError_t expert_sort_launch(const void *ids, int64_t ld_ids, bool wide, int64_t tokens, int64_t k,
                               int64_t experts, int32_t *position, int32_t *offsets,
                               void *workspace, int *launches, cudaStream_t s) {
  SortParams p{};
  p.ids = ids, p.ld_ids = ld_ids, p.wide = wide;
  p.n = tokens * k;
  p.k = static_cast<int32_t>(std::max<int64_t>(k, 1));
  p.experts = static_cast<int32_t>(experts);
  const int64_t chunk = chunk_of(p.n);
  const int64_t chunks = std::max<int64_t>((p.n + chunk - 1) / chunk, 1);
  p.chunk = static_cast<int32_t>(chunk), p.chunks = static_cast<int32_t>(chunks);
  p.position = position, p.offsets = offsets;
  p.counts = static_cast<int32_t *>(workspace);
  const dim3 grid(static_cast<unsigned>(chunks));
  *launches = 0;
  if (chunks > 1) {
    launch_pdl(expert_count_kernel, grid, kSortThreads, experts * sizeof(int32_t), s, p);
    *launches += 1;
  }
  const size_t smem = static_cast<size_t>(2 + kSortWarps) * experts * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>((2 + kSortWarps) * kMaxExperts * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  launch_pdl(expert_place_kernel, grid, kSortThreads, smem, s, p);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace ff
}  // namespace gemm_gb300
