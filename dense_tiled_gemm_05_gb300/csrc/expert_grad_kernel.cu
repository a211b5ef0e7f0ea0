// expert_grad_kernel.cu -- the gradients of the experts' weights: for each expert e and the rows
// r in [offsets[e], offsets[e + 1]),
//
//   D[e] = sum_r A[r]^T B[r]
//
// (A: rows x MA, B: rows x NB, D: experts x MA x NB). Both operands have the sum's axis outside
// and are read in place, MN-major: a CTA pair's 256 x 256 tile takes 64 rows a K-block.
//
// An expert's rows end anywhere. TMA fills what lies outside the matrices with zeros, but the
// rows after an expert's last are the next expert's (or nothing's: they may hold NaN), so they
// have to leave both operands. The MMAs of the last K-block stop at the 16-row step that holds
// the last row; of that step the up to 15 rows past it are set to zero in shared memory, by a
// warp that the block's copies wait for instead of the MMA issuer (its own barrier), and that then
// tells the issuer. All other blocks go from TMA to the MMAs as ever.
//
// The schedule is fixed, tile by tile through the experts, so that the clusters at work read the
// same rows from L2, each from another K-block on (all from the first: 4 to 9 % slower). Tiles of an
// expert with many rows run long: the experts come in the order of their rows, most first, and every
// other round of clusters runs backwards, so that the shares even out (16 experts of 46 to 4407
// rows, 2048 x 4096: 184 us, 189 in their own order; 64 experts of 0 to 1781 rows, 1024 x 2048: 81
// and 84). An expert without rows gets zeros. One accumulation a tile, in a fixed order: the same
// call gives the same bits. Bound by the tensor cores for many rows an expert (16384 rows,
// 4096 x 2048: one expert 1730 TFLOP/s, 16 of 1024 rows 1690 to 1730), by the writing of D for few (64
// of 256 rows: 244 us for 1.07 GB written and 0.2 read). A tile's rows are not shared over clusters:
// fewer tiles than those leave them idle (5 experts of 4564 rows, 488 x 112: ten tiles, 29 us).
#include "activation.cuh"
#include "expert_kernels.h"
#include "expert_tiles.cuh"
#include "ff_boxes.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

using namespace tc;

constexpr int BM = 128;                         // columns of A per CTA
constexpr int BN = 256;
constexpr int BK = 64;                          // rows a K-block
constexpr int PANEL_BYTES = BK * kRowBytes;     // 64 columns of 64 rows
constexpr int PANELS = 4;                       // two of A, two of B
constexpr int STAGE_BYTES = PANELS * PANEL_BYTES;
constexpr int STAGES = 5;
constexpr int kEpi = 8;                         // epilogue warps
constexpr int kMaskWarp = 2 + kEpi;
constexpr int kGradThreads = 32 * (kMaskWarp + 1);
constexpr int HALF = BN / 2;                    // accumulator columns of an epilogue warp
constexpr int EPI_OFFSET = STAGES * STAGE_BYTES;
constexpr int BAR_OFFSET = EPI_OFFSET + kEpi * 2 * kStoreBufBytes;
constexpr int SMEM_BYTES = 232448;              // (all of it: see expert_pair_kernel.cu)
constexpr int ORDER_OFFSET = BAR_OFFSET + (4 * STAGES + 5) * 8 + (8 + 2 * STAGES) * 4;
constexpr int kOrdered = 256;                   // experts that are put in order, at most
static_assert(ORDER_OFFSET + (kOrdered + 1) * 4 + kOrdered + 1024 <= SMEM_BYTES, "shared memory");

// Experts by their rows, most first (equal ones by number), and their first rows, in shared memory,
// where a tile's place takes each role 400 cycles to find. More experts than kOrdered come in their
// own order, from global memory. Offsets are kept inside [0, rows], and an expert whose end lies
// before its start has no rows.
struct ExpertOrder {
  int32_t *offsets;  // [kOrdered + 1]
  uint8_t *order;    // [kOrdered]
  bool here;
  // by all threads; a barrier has to follow
  __device__ __forceinline__ void fill(const ExpertGradParams &p) const {
    if (!here) return;
    for (int e = threadIdx.x; e <= p.experts; e += kGradThreads)
      offsets[e] = max(0, min(p.offsets[e], p.rows));
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kGradThreads) {
      const int n = offsets[e + 1] - offsets[e];
      int rank = 0;
      for (int i = 0; i < p.experts; ++i) {
        const int m = offsets[i + 1] - offsets[i];
        rank += m > n || (m == n && i < e);
      }
      order[rank] = static_cast<uint8_t>(e);
    }
  }
  __device__ __forceinline__ int at(int i) const { return here ? order[i] : i; }
  __device__ __forceinline__ void rows_of(const ExpertGradParams &p, int e, int &lo, int &n) const {
    lo = here ? offsets[e] : max(0, min(p.offsets[e], p.rows));
    const int hi = here ? offsets[e + 1] : max(0, min(p.offsets[e + 1], p.rows));
    n = max(hi - lo, 0);
  }
};

// A tile of an expert: its rows and columns.
struct Tile {
  int e, lo, blocks, last;  // first row, K-blocks, rows of the last block
  int start;                // the K-block that the sum begins with; it wraps after the last one
  int m0, n0;
  __device__ __forceinline__ Tile(const ExpertGradParams &p, const ExpertOrder &order, int t) {
    const int per = p.tiles_m * p.tiles_n;
    const int place = static_cast<uint32_t>(t) / static_cast<uint32_t>(per), i = t - place * per;
    e = order.at(place);
    n0 = static_cast<uint32_t>(i) / static_cast<uint32_t>(p.tiles_m);
    m0 = (i - n0 * p.tiles_m) * (2 * BM);
    n0 *= BN;
    int n;
    order.rows_of(p, e, lo, n);
    blocks = (n + BK - 1) / BK;
    last = n - (blocks - 1) * BK;
    // (neighbouring tiles start apart, at multiples of what a power of two below `blocks` allows)
    start = blocks > 0 ? i & ((1 << (31 - __clz(blocks))) - 1) : 0;
  }
  __device__ __forceinline__ bool ragged() const { return blocks > 0 && last % 16 != 0; }
};

// A cluster's tiles: one of every round, forwards and backwards in turn.
struct Rounds {
  int cluster, clusters, tiles, i;
  __device__ __forceinline__ bool next(int &t) {
    t = i * clusters + (i & 1 ? clusters - 1 - cluster : cluster);
    ++i;
    return t < tiles;
  }
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, uint32_t src, int32_t x, int32_t y,
                                             int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// 128 columns of 64 rows of an operand, as two panels.
__device__ __forceinline__ void load_panels(uint32_t dst, const CUtensorMap *m, int one, uint32_t bar,
                                            int col, int row, uint64_t policy) {
  if (one) {
    tma_load_3d_pair_hint(dst, m, bar, 0, row, col / 64, policy);
  } else {
    tma_load_2d_pair_hint(dst, m, bar, col, row, policy);
    tma_load_2d_pair_hint(dst + PANEL_BYTES, m, bar, col + 64, row, policy);
  }
}

// This warp's 32 rows and 128 columns of the tile: by TMA through its two boxes, ...
template <int OUT>
__device__ __forceinline__ void store_boxes(const CUtensorMap *tmD, const ExpertGradParams &p, uint32_t t_row,
                                            bool zero, uint8_t *boxes, int &next, int lane, int row0,
                                            int n0, int e) {
  if (row0 >= p.MA) return;
#pragma unroll 1
  for (int c = 0; c < HALF && n0 + c < p.NB; c += 64) {
    float v[64];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = 0.0f;
    } else {
      read_columns<64>(t_row + c, v);
    }
    uint8_t *box = boxes + next * kStoreBufBytes;
    next ^= 1;
    if (lane == 0) bulk_wait_group_read<1>();  // the store that last used this box has read it
    __syncwarp();
    write_box_row<OUT>(smem_u32(box) + lane * kRowBytes, lane, v);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(tmD, smem_u32(box), n0 + c, row0, e);
      bulk_commit_group();
    }
  }
}
// ... or, where TMA cannot address D, by rows: a warp's 32 x 32 values turn in shared memory, so that
// the lanes of a store are neighbours (2048 x 1001 of 32 experts, all rows unaligned: 70 us; with a row a
// lane and slower copies of the operands 565).
template <typename T>
__device__ __forceinline__ void store_direct(const ExpertGradParams &p, uint32_t t_row, bool zero, uint8_t *box,
                                             int lane, int row0, int n0, int e) {
  constexpr int PITCH = 34;  // 17 words a row: neither side meets a bank twice
  T *turn = reinterpret_cast<T *>(box);
  const int rows = min(32, p.MA - row0);
  if (rows <= 0) return;
#pragma unroll 1
  for (int c = 0; c < HALF && n0 + c < p.NB; c += 32) {
    float v[32];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    } else {
      read_columns<32>(t_row + c, v);
    }
    __syncwarp();  // the previous columns have been read
#pragma unroll
    for (int i = 0; i < 32; ++i) turn[lane * PITCH + i] = from_f32<T>(v[i]);
    __syncwarp();
    T *d = static_cast<T *>(p.D) + e * p.stride_d + row0 * p.ldd + n0 + c + lane;
    if (n0 + c + lane < p.NB)
      for (int r = 0; r < rows; ++r) d[r * p.ldd] = turn[r * PITCH + lane];
  }
}

__global__ void __launch_bounds__(kGradThreads, 1)
    expert_grad_kernel(const __grid_constant__ ExpertGradMaps maps, const ExpertGradParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + BAR_OFFSET);
  uint64_t *empty = full + STAGES;
  uint64_t *tail = empty + STAGES;     // a ragged block's copies, this CTA's own
  uint64_t *masked = tail + STAGES;    // (the leader's) both CTAs' surplus rows are zero
  uint64_t *tmem_full = masked + STAGES;
  uint64_t *tmem_empty = tmem_full + 2;
  uint64_t *drain = tmem_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  // Teardown words, as in expert_pair_kernel.cu.
  volatile uint32_t *xs = reinterpret_cast<volatile uint32_t *>(tmem_slot + 2);
  volatile uint32_t *fill_bytes = xs + 4, *peer_bytes = fill_bytes + STAGES;
  // stages whose own barriers were used for ragged blocks, and the parities of their last uses
  volatile uint32_t *tails = peer_bytes + STAGES;

  const int warp = uniform(static_cast<int>(threadIdx.x / 32));
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
      mbar_init(&masked[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], 2 * kEpi);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    for (int i = 0; i < 6 + 2 * STAGES; ++i) xs[i] = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.A);
    prefetch_tensormap(&maps.B);
    if (p.tma_out) prefetch_tensormap(&maps.D);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));
  const uint32_t smem_base = smem_u32(smem);
  // Up to here only this CTA's own resources: the prologue may overlap the previous kernel.
  grid_dependency_wait();
  grid_launch_dependents();
  const ExpertOrder order{reinterpret_cast<int32_t *>(smem + ORDER_OFFSET),
                          smem + ORDER_OFFSET + (kOrdered + 1) * 4, p.experts <= kOrdered};
  order.fill(p);
  __syncthreads();
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  Rounds rounds{static_cast<int>(blockIdx.x / 2), static_cast<int>(gridDim.x / 2),
                p.experts * p.tiles_m * p.tiles_n, 0};
  int t;

  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    // (the whole warp walks, one lane issues)
    const bool issuer = elect_one();
    uint32_t stage = 0, phase = 0, issued = 0;
    uint32_t tail_used = 0, tail_parity = 0;  // by stage: used at all, parity of the last use
    bool ok = (p.debug_flags & kDebugStallProducer) == 0;
    const int stop_after = stall_after_fills(p.debug_flags, static_cast<int>(rank));
    const uint64_t keep = l2_policy_evict_last();
    const uint32_t full_bars = mapa_shared(smem_u32(full), 0);  // the leader's
    const uint32_t tail_bars = mapa_shared(smem_u32(tail), rank);
    while (ok && rounds.next(t)) {
      const Tile tile(p, order, t);
      const int m0 = uniform(tile.m0) + static_cast<int>(rank) * BM;
      const int n0 = uniform(tile.n0) + static_cast<int>(rank) * BM;
      const int blocks = uniform(tile.blocks), first = uniform(tile.lo);
      const int own_block = uniform(tile.ragged() ? tile.blocks - 1 : -1);
      int kb = uniform(tile.start);
      for (int i = 0; i < blocks; ++i) {
        if (stop_after >= 0 && issued >= static_cast<uint32_t>(stop_after)) {
          ok = false;  // test hook: this loader stops here, copies still in flight
          break;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1, wd));
        if (!ok) break;
        const bool own = kb == own_block;
        if (own) {
          tail_parity = tail_used >> stage & 1 ? tail_parity ^ 1u << stage : tail_parity & ~(1u << stage);
          tail_used |= 1u << stage;
        }
        if (issuer) {
          const uint32_t fb = (own ? tail_bars : full_bars) + stage * 8;
          if (own) {
            mbar_arrive_expect_tx(&tail[stage], STAGE_BYTES);
            if (leader) mbar_arrive(&full[stage]);
          } else if (leader) {
            mbar_arrive_expect_tx(&full[stage], 2u * STAGE_BYTES);
          }
          fill_bytes[stage] = own ? 0 : STAGE_BYTES;
          const uint32_t dst = smem_base + stage * STAGE_BYTES;
          load_panels(dst, &maps.A, p.panels_a, fb, m0, first + kb * BK, keep);
          load_panels(dst + 2 * PANEL_BYTES, &maps.B, p.panels_b, fb, n0, first + kb * BK, keep);
        }
        __syncwarp();
        ++issued;
        if (++kb == blocks) kb = 0;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) {
      xs[0] = issued;
      tails[0] = tail_used;
      tails[1] = tail_parity;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer (leader)
    if (leader) {  // (the whole warp walks, one lane issues)
      const bool issuer = elect_one();
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, consumed = 0, masked_phase = 0;
      bool ok = true;
      while (ok && rounds.next(t)) {
        const Tile tile(p, order, t);
        const int blocks = uniform(tile.blocks);
        if (blocks == 0) continue;
        const int last = uniform(tile.last);
        const bool ragged = last % 16 != 0;
        int kb = uniform(tile.start);
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_empty[acc], acc_phase ^ 1, wd));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int i = 0; i < blocks; ++i) {
          const bool end = kb == blocks - 1;
          ok = mbar_wait(&full[stage], phase, wd);
          if (end && ragged) {
            ok = ok && mbar_wait_cluster(&masked[stage], masked_phase >> stage & 1, wd);
            masked_phase ^= 1u << stage;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++consumed;
          tc_fence_after();
          const uint32_t a_base = smem_base + stage * STAGE_BYTES;
          const uint64_t ad = sdesc_sw128(a_base, PANEL_BYTES, 1024);
          const uint64_t bd = sdesc_sw128(a_base + 2 * PANEL_BYTES, PANEL_BYTES, 1024);
          const int steps = end ? (last + 15) / 16 : BK / 16;
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)  // (16 rows on: 2048 bytes, in units of 16)
              if (kk < steps)
                mma_f16_pair(d_tmem, ad + kk * (16 * kRowBytes / 16), bd + kk * (16 * kRowBytes / 16), p.idesc,
                             i != 0 || kk != 0);
            mma_commit_pair_multicast(&empty[stage], 0x3);
          }
          __syncwarp();
          if (++kb == blocks) kb = 0;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (issuer) mma_commit_pair_multicast(&tmem_full[acc], 0x3);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (issuer) {
        mma_commit_pair(drain);
        drain_wait(drain, 0, p.timeout_ns);
        xs[1] = consumed;
      }
    }
    __syncwarp();
  } else if (warp == kMaskWarp) {
    // ------------------------- rows past an expert's last: zeros (both CTAs)
    // (a wait spans all tiles since the last ragged one, and so has their limits together: should one
    // of them stop, the role that waits for it raises the abort flag, which ends this wait too)
    uint32_t fills = 0, phases = 0;
    Watchdog patient = wd;
    for (patient.timeout_ns = 0; rounds.next(t);) {
      const Tile tile(p, order, t);
      const uint32_t before = fills;
      fills += static_cast<uint32_t>(tile.blocks);
      if (patient.timeout_ns >> 62 == 0) patient.timeout_ns += wd.timeout_ns;
      if (!tile.ragged()) continue;
      const uint32_t stage = (before + static_cast<uint32_t>(tile.blocks - 1 - tile.start)) % STAGES;
      bool ok = mbar_wait(&tail[stage], phases >> stage & 1, patient);
      patient.timeout_ns = 0;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      phases ^= 1u << stage;
      const int first = tile.last, n = (tile.last + 15) / 16 * 16 - first;
      // 8 pieces of 16 bytes a row and panel (a row is zero whatever its swizzle)
      for (int i = lane; i < n * PANELS * 8; i += 32) {
        const int piece = i % 8, panel = i / 8 % PANELS, row = first + i / (8 * PANELS);
        *reinterpret_cast<uint4 *>(smem + stage * STAGE_BYTES + panel * PANEL_BYTES + row * kRowBytes +
                                   piece * 16) = uint4{0, 0, 0, 0};
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&masked[stage]), 0));
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;
    const int e = warp - 2;
    const int half = e / 4;
    uint8_t *boxes = smem + EPI_OFFSET + e * 2 * kStoreBufBytes;
    int next = 0;
    uint32_t acc = 0, acc_phase = 0;
    while (rounds.next(t)) {
      const Tile tile(p, order, t);
      const bool zero = tile.blocks == 0;
      if (!zero) {
        bool ok = mbar_wait_cluster(&tmem_full[acc], acc_phase, wd);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN + half * HALF;
      const int row0 = tile.m0 + static_cast<int>(rank) * BM + quarter * 32, n0 = tile.n0 + half * HALF;
      if (p.tma_out) {
        if (p.dtype == GEMM_BF16)
          store_boxes<GEMM_BF16>(&maps.D, p, t_row, zero, boxes, next, lane, row0, n0, tile.e);
        else
          store_boxes<GEMM_F16>(&maps.D, p, t_row, zero, boxes, next, lane, row0, n0, tile.e);
      } else if (p.dtype == GEMM_BF16) {
        store_direct<__nv_bfloat16>(p, t_row, zero, boxes, lane, row0, n0, tile.e);
      } else {
        store_direct<__half>(p, t_row, zero, boxes, lane, row0, n0, tile.e);
      }
      if (zero) continue;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_read(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&xs[3])), rank ^ 1u),
                          *abort_flag ? 1u : 0u);
    if (!leader) {
      st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&xs[2])), 0), xs[0]);
      for (int s = 0; s < STAGES; ++s)
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&peer_bytes[s])), 0),
                              fill_bytes[s]);
    }
  }
  tc_fence_before();
  cluster_sync();
  if (*abort_flag || xs[3]) {
    if (threadIdx.x == 0)
      for (int i = 0; i < STAGES; ++i)
        if (tails[0] >> i & 1) drain_wait(&tail[i], tails[1] >> i & 1, p.timeout_ns);
    if (leader && threadIdx.x == 0)
      drain_sized_fills<STAGES>(full, xs[1], xs[0], xs[2], fill_bytes, peer_bytes, p.timeout_ns);
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * BN);
  }
}

}  // namespace

cudaError_t expert_grad_launch(const ExpertGradMaps &maps, const ExpertGradParams &p, int grid,
                               cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(expert_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dependency_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kGradThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, expert_grad_kernel, maps, p);
}

}  // namespace ff
}  // namespace gemm_gb300
