// ff_pair_kernel.cu -- products of many tokens with an epilogue, and the gated pair:
//
//   Y = act(X W (+ X2 W2) + bias) + residual      or      H = act(X Wg) * (X Wu)
//
// The tile machinery is the CTA-pair product kernel's (tc2_kernel.cu): a cluster of two CTAs
// on two SMs computes a 256 x 256 fp32 accumulator with tcgen05.mma.cta_group::2, two
// accumulators alternate in TMEM so that one tile's epilogue runs under the next tile's
// K-loop, and the last, partly filled rounds of tiles are split along K (sk_schedule.h).
//
// Each CTA of a pair loads half of the accumulator's columns of weights. For the gated
// product the halves come from different matrices: the leader loads 128 rows of the gate's
// weights, the peer the same 128 rows of the up projection's. One MMA then forms g in columns
// 0-127 and u in columns 128-255 of the same rows, every epilogue thread finds both of its
// row in its own TMEM lane, and X is read once for both products.
//
// A sum of two products walks the first pair's K-blocks and then the second's into the same
// accumulator: one fp32 sum, one rounding.
//
// The epilogue replaces the product's round trip through memory (a 4-byte write and read per
// output element plus a launch): per 64 columns a warp reads its 32 rows from TMEM, applies
// bias (staged in shared memory), activation and residual (loaded by TMA into the box the
// result is then written over), and stores 32 x 128-byte boxes by TMA.
#include "activation.cuh"
#include "ff_kernels.h"
#include "tc_common.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

using namespace tc;

constexpr int BM = kTcBlockM;                 // rows per CTA
constexpr int BN = 256;                       // accumulator columns
constexpr int BK = 64;
constexpr int A_BYTES = BM * kRowBytes;
constexpr int B_BYTES = (BN / 2) * kRowBytes;
constexpr int PANEL_BYTES = BK * kRowBytes;   // MN-major weights: 64 K-rows x 128 bytes
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
// Eight epilogue warps, two for each quarter of the TMEM lanes, each with half of the
// accumulator's columns: four left each scheduler one warp, whose exponentials, TMEM reads and
// TMA waits then ran one after another (silu and a residual took 8 us a tile). Their boxes
// leave room for five stages.
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int HALF = BN / 2;                  // accumulator columns of an epilogue warp
constexpr int STAGES = 5;
constexpr int EPI_OFFSET = STAGES * STAGE_BYTES;
constexpr int BIAS_OFFSET = EPI_OFFSET + kPairEpiWarps * 2 * kStoreBufBytes;
constexpr int BAR_OFFSET = BIAS_OFFSET + kPairEpiWarps * 32 * 4;
constexpr int PART_BYTES = HALF * 32 * 4;     // one partial's 32 rows of a warp, fp32
// stages, accumulators, drain; per epilogue warp one partial load and two residual boxes
constexpr int NUM_BARS = 2 * STAGES + 5 + kPairEpiWarps * 3;
constexpr int SMEM_BYTES = BAR_OFFSET + NUM_BARS * 8 + 32 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert(kPairEpiWarps * PART_BYTES <= STAGES * STAGE_BYTES, "owners' partials fit the stages");

// COLS consecutive accumulator columns of this lane's row, as fp32. By whole warps, whose lanes
// may come from rows past M or from a store that one of them issued.
template <int COLS>
__device__ __forceinline__ void read_columns(uint32_t taddr, float (&v)[COLS]) {
  __syncwarp();
  uint32_t r[COLS / 32][32];
#pragma unroll
  for (int h = 0; h < COLS / 32; ++h) tmem_ld_32x32b_x32(taddr + h * 32, r[h]);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < COLS; ++i) v[i] = __uint_as_float(r[i / 32][i % 32]);
}

// One row of a 32-row, 128-byte-wide box (128-byte swizzle): v rounded to OUT.
template <int OUT, int COLS>
__device__ __forceinline__ void write_box_row(uint32_t row_addr, int lane, const float (&v)[COLS]) {
  constexpr int PER = OUT == GEMM_F32 ? 4 : 8;  // elements in 16 bytes
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = OUT == GEMM_F32 ? __float_as_uint(v[ch * PER + i])
                             : pack2<OUT>(__float_as_uint(v[ch * PER + 2 * i]),
                                          __float_as_uint(v[ch * PER + 2 * i + 1]));
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + ((ch ^ (lane & 7)) << 4)),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
}

// v += the 8 (4) elements of type OUT in 16 bytes.
template <int OUT>
__device__ __forceinline__ void add_chunk(float *v, uint4 w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (OUT == GEMM_F32) {
      v[i] += __uint_as_float(x[i]);
    } else if (OUT == GEMM_BF16) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x[i]));
      v[2 * i] += f.x, v[2 * i + 1] += f.y;
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
      v[2 * i] += f.x, v[2 * i + 1] += f.y;
    }
  }
}

template <int OUT, int COLS>
__device__ __forceinline__ void add_box_row(uint32_t row_addr, int lane, float (&v)[COLS]) {
  constexpr int PER = OUT == GEMM_F32 ? 4 : 8;
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(row_addr + ((ch ^ (lane & 7)) << 4))
                 : "memory");
    add_chunk<OUT>(&v[ch * PER], w);
  }
}

// A warp's two staging boxes and the residual loads into them.
struct Boxes {
  uint8_t *mem;         // two boxes of kStoreBufBytes
  float *bias;          // 32 floats
  uint64_t *bars;       // residual load of each box
  uint32_t phases;      // their parities
  int next;             // box of the next store
  int lane;

  __device__ __forceinline__ uint8_t *box(int b) const { return mem + b * kStoreBufBytes; }
  __device__ __forceinline__ uint32_t row(int b) const { return smem_u32(box(b)) + lane * kRowBytes; }
  // The next box to write, once the store that last used it has read it.
  __device__ __forceinline__ int take() {
    if (lane == 0) bulk_wait_group_read<1>();
    __syncwarp();
    const int b = next;
    next ^= 1;
    return b;
  }
  __device__ __forceinline__ void store(int b, const CUtensorMap *m, int x, int y) const {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(m, smem_u32(box(b)), x, y);
      bulk_commit_group();
    }
  }
  __device__ __forceinline__ void load(int b, const CUtensorMap *m, int x, int y) const {
    if (lane == 0) {
      bulk_wait_group_read<0>();
      mbar_arrive_expect_tx(&bars[b], kStoreBufBytes);
      tma_load_2d(smem_u32(box(b)), m, smem_u32(&bars[b]), x, y);
    }
  }
};

// Whether this tile's residual comes through the boxes (the pre-activation, when it is kept,
// needs both boxes for stores).
__device__ __forceinline__ bool residual_boxes(const PairParams &p) {
  return p.tma_out && p.f.residual && !p.f.pre;
}
template <int OUT>
__device__ __forceinline__ int box_count(const PairParams &p, int row0, int n0, int cols) {
  constexpr int COLS = OUT == GEMM_F32 ? 32 : 64;
  return row0 >= p.f.M || n0 >= p.f.N ? 0 : (min(cols, p.f.N - n0) + COLS - 1) / COLS;
}

// Plain product, TMA form.
template <int OUT>
__device__ __forceinline__ bool plain_boxes(const PairMaps &maps, const PairParams &p, Boxes &bx,
                                            uint32_t t_row, int row0, int n0, const Watchdog &wd) {
  constexpr int COLS = OUT == GEMM_F32 ? 32 : 64;
  const int lane = bx.lane;
  const int n = box_count<OUT>(p, row0, n0, HALF);
  const bool res_box = residual_boxes(p);
  float b0 = 0.0f, b1 = 0.0f;  // the next piece's bias, two columns a lane
  auto load_bias = [&](int c) {
    const int j = n0 + c * COLS + lane;
    b0 = c < n && j < p.f.N ? load_any(p.f.bias, p.f.bias_dtype, j) : 0.0f;
    if (COLS == 64) b1 = c < n && j + 32 < p.f.N ? load_any(p.f.bias, p.f.bias_dtype, j + 32) : 0.0f;
  };
  if (p.f.bias) load_bias(0);
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    const int col = n0 + c * COLS;
    float v[COLS];
    read_columns<COLS>(t_row + c * COLS, v);
    if (p.f.bias) {
#pragma unroll
      for (int h = 0; h < COLS / 32; ++h) {
        __syncwarp();  // the previous columns' bias has been read
        bx.bias[lane] = h ? b1 : b0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 q = *reinterpret_cast<const float4 *>(bx.bias + i);
          float *o = &v[32 * h + i];
          o[0] += q.x, o[1] += q.y, o[2] += q.z, o[3] += q.w;
        }
      }
      load_bias(c + 1);
    }
    if (p.f.pre) {
      const int b = bx.take();
      write_box_row<OUT>(bx.row(b), lane, v);
      bx.store(b, &maps.Z, col, row0);
    }
    activate_all<true>(v, p.f.act);
    if (res_box) {
      const int b = c & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&bx.bars[b], (bx.phases >> b) & 1u, wd))) return false;
      bx.phases ^= 1u << b;
      add_box_row<OUT>(bx.row(b), lane, v);
      write_box_row<OUT>(bx.row(b), lane, v);
      bx.store(b, &maps.C, col, row0);
      bx.next = b ^ 1;  // (a split tile's partial may follow, through the other box first)
      if (c + 2 < n) bx.load(b, &maps.R, col + 2 * COLS, row0);
      continue;
    }
    if (p.f.residual && row0 + lane < p.f.M) {
      constexpr int PER = OUT == GEMM_F32 ? 4 : 8;
      constexpr int ES = OUT == GEMM_F32 ? 4 : 2;
      const char *r = static_cast<const char *>(p.f.residual) +
                      ((row0 + lane) * p.f.ld_residual + col) * ES;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)  // (a row of the output ends on a 16-byte boundary)
        if (col + ch * PER < p.f.N) add_chunk<OUT>(&v[ch * PER], *reinterpret_cast<const uint4 *>(r + ch * 16));
    }
    const int b = bx.take();
    write_box_row<OUT>(bx.row(b), lane, v);
    bx.store(b, &maps.C, col, row0);
  }
  return true;
}

// Gated pair, TMA form: 64 columns of g and, 128 accumulator columns on, of u.
template <int OUT>
__device__ __forceinline__ void gated_boxes(const PairMaps &maps, const PairParams &p, Boxes &bx,
                                            uint32_t t_row, int row0, int col) {
  constexpr int COLS = HALF / 2;
  const int lane = bx.lane;
  if (box_count<OUT>(p, row0, col, COLS) == 0) return;
  float g[COLS], u[COLS];
  read_columns<COLS>(t_row, g);
  if (p.f.pre) {
    const int b = bx.take();
    write_box_row<OUT>(bx.row(b), lane, g);
    bx.store(b, &maps.Z, col, row0);
  }
  read_columns<COLS>(t_row + BN / 2, u);
  if (p.f.pre) {
    const int b = bx.take();
    write_box_row<OUT>(bx.row(b), lane, u);
    bx.store(b, &maps.Z2, col, row0);
  }
  activate_all<true>(g, p.f.act);
#pragma unroll
  for (int i = 0; i < COLS; ++i) g[i] *= u[i];
  const int b = bx.take();
  write_box_row<OUT>(bx.row(b), lane, g);
  bx.store(b, &maps.C, col, row0);
}

// Outputs or a residual TMA cannot address: each lane reads and writes its row's elements.
template <typename T, bool GATED>
__device__ __forceinline__ void direct_rows(const PairParams &p, uint32_t t_row, int row, int n0) {
  const int cols = GATED ? HALF / 2 : HALF;  // this warp's
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 32) {
    float v[32], u[32];
    read_columns<32>(t_row + c0, v);
    if (GATED) read_columns<32>(t_row + BN / 2 + c0, u);
    const int col = n0 + c0;
    if (row >= p.f.M || col >= p.f.N) continue;
    const int n = min(32, p.f.N - col);
    if (!GATED && p.f.bias) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) v[j] += load_any(p.f.bias, p.f.bias_dtype, col + j);
    }
    if (p.f.pre) {
      T *z = static_cast<T *>(p.f.pre) + row * p.f.ld_pre + col;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) z[j] = from_f32<T>(v[j]);
      if (GATED) {
        T *z2 = static_cast<T *>(p.f.pre2) + row * p.f.ld_pre2 + col;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n) z2[j] = from_f32<T>(u[j]);
      }
    }
    activate_all<true>(v, p.f.act);
    if (GATED) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= u[j];
    } else if (p.f.residual) {
      const T *r = static_cast<const T *>(p.f.residual) + row * p.f.ld_residual + col;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) v[j] += to_f32(r[j]);
    }
    T *y = static_cast<T *>(p.f.C) + row * p.f.ldc + col;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) y[j] = from_f32<T>(v[j]);
  }
}

template <bool GATED, bool W_MN>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + BAR_OFFSET);
  uint64_t *empty = full + STAGES;
  uint64_t *tmem_full = empty + STAGES;
  uint64_t *tmem_empty = tmem_full + 2;
  uint64_t *drain = tmem_empty + 2;
  uint64_t *part_bar = drain + 1;                  // [kPairEpiWarps]
  uint64_t *res_bar = part_bar + kPairEpiWarps;    // [kPairEpiWarps][2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(res_bar + 2 * kPairEpiWarps);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  // Teardown words, as in tc2_kernel.cu: fills this CTA's loader issued, fills the MMA issuer
  // consumed, fills the peer's loader issued, whether the other CTA aborted.
  volatile uint32_t *xs = reinterpret_cast<volatile uint32_t *>(tmem_slot + 2);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  constexpr int TILE_N = GATED ? BN / 2 : BN;  // output columns per tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], 2 * kPairEpiWarps);
    }
    mbar_init(drain, 1);
    for (int w = 0; w < 3 * kPairEpiWarps; ++w) mbar_init(&part_bar[w], 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) xs[i] = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.X);
    prefetch_tensormap(&maps.W);
    if (p.tma_out) prefetch_tensormap(&maps.C);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Up to here only this CTA's own resources: the prologue may overlap the previous kernel.
  grid_dependency_wait();
  grid_launch_dependents();
  const Watchdog wd{abort_flag, p.f.status, p.f.timeout_ns};
  const int cluster_id = blockIdx.x / 2;
  const SkSchedule sched =
      sk_make(p.tiles_m * p.tiles_n, p.f.k_blocks, gridDim.x / 2, p.sk_dp_tiles);
  const bool split = p.sk_dp_tiles < p.tiles_m * p.tiles_n;
  const int epoch = split ? sk_epoch_begin(p.sk_epoch_word) : 0;

  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, issued = 0;
      bool ok = (p.f.debug_flags & kDebugStallProducer) == 0;
      const int stop_after = stall_after_fills(p.f.debug_flags, static_cast<int>(rank));
      const uint64_t keep = l2_policy_evict_last();  // operand tiles outlive the outputs in L2
      WorkIter work(sched, cluster_id);
      SkSegment seg;
      while (ok && work.next(seg)) {
        int pm, pn;
        tile_coords(seg.tile, p.tiles_m, p.tiles_n, p.group_m, pm, pn);
        const int m0 = pm * (2 * BM) + static_cast<int>(rank) * BM;
        const int n0 = GATED ? pn * TILE_N : pn * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = seg.kb_begin; kb < seg.kb_end; ++kb) {
          if (stop_after >= 0 && issued >= static_cast<uint32_t>(stop_after)) {
            ok = false;  // test hook: this loader stops here, copies still in flight
            break;
          }
          if (!mbar_wait(&empty[stage], phase ^ 1, wd)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * STAGE_BYTES);
          const uint32_t a_dst = smem_u32(smem + stage * STAGE_BYTES);
          const uint32_t b_dst = a_dst + A_BYTES;
          const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);  // the leader's barrier
          const bool second = !GATED && kb >= p.f.kb_first;
          const int k0 = (second ? kb - p.f.kb_first : kb) * BK;
          tma_load_2d_pair_hint(a_dst, second ? &maps.X2 : &maps.X, fb, k0, m0, keep);
          const CUtensorMap *w = (GATED ? !leader : second) ? &maps.W2 : &maps.W;
          if (W_MN) {
            tma_load_2d_pair_hint(b_dst, w, fb, n0, k0, keep);
            tma_load_2d_pair_hint(b_dst + PANEL_BYTES, w, fb, n0 + 64, k0, keep);
          } else {
            tma_load_2d_pair_hint(b_dst, w, fb, k0, n0, keep);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      xs[0] = issued;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer (leader)
    if (leader && lane == 0) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, consumed = 0;
      bool ok = true;
      WorkIter work(sched, cluster_id);
      SkSegment seg;
      while (ok && work.next(seg)) {
        if (!mbar_wait_cluster(&tmem_empty[acc], acc_phase ^ 1, wd)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = seg.kb_begin; kb < seg.kb_end; ++kb) {
          if (!mbar_wait(&full[stage], phase, wd)) {
            ok = false;
            break;
          }
          ++consumed;
          tc_fence_after();
          const uint32_t a_base = smem_u32(smem + stage * STAGE_BYTES);
          const uint32_t b_base = a_base + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = sdesc_sw128(a_base + kk * 32, 16, 1024);
            const uint64_t bd = W_MN ? sdesc_sw128(b_base + kk * 16 * kRowBytes, PANEL_BYTES, 1024)
                                     : sdesc_sw128(b_base + kk * 32, 16, 1024);
            mma_f16_pair(d_tmem, ad, bd, p.f.idesc, (kb != seg.kb_begin) || kk != 0);
          }
          mma_commit_pair_multicast(&empty[stage], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_pair_multicast(&tmem_full[acc], 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      mma_commit_pair(drain);
      drain_wait(drain, 0, p.f.timeout_ns);
      xs[1] = consumed;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;
    const int e = warp - 2;
    const int half = e / 4;  // its columns: of the accumulator, and (gated: halved) of the tile
    const int out_half = half * TILE_N / 2;
    Boxes bx{smem + EPI_OFFSET + e * 2 * kStoreBufBytes,
             reinterpret_cast<float *>(smem + BIAS_OFFSET) + e * 32, res_bar + 2 * e, 0, 0, lane};
    // The accumulator columns a warp hands over or joins are those its epilogue reads: half of
    // them, or half of g's and half of u's.
    constexpr int PARTS = GATED ? 2 : 1, PART_COLS = HALF / PARTS;
    auto part_col = [&](int i) { return i * (BN / 2) + half * PART_COLS; };
    uint32_t acc = 0, acc_phase = 0, part_phase = 0;
    WorkIter work(sched, cluster_id);
    SkSegment seg;
    bool ok = true;
    int loads = 0;  // residual loads in flight when the loop ends early
    while (ok && work.next(seg)) {
      int pm, pn;
      tile_coords(seg.tile, p.tiles_m, p.tiles_n, p.group_m, pm, pn);
      const int row0 = pm * (2 * BM) + static_cast<int>(rank) * BM + quarter * 32;
      const int n0 = pn * TILE_N + out_half;
      if (!GATED && seg.role != kSegPartial && residual_boxes(p)) {
        // the first two pieces of the residual, ahead of the accumulator
        const int cols = p.f.out_dtype == GEMM_F32 ? 32 : 64;
        loads = p.f.out_dtype == GEMM_F32 ? box_count<GEMM_F32>(p, row0, n0, HALF)
                                          : box_count<GEMM_BF16>(p, row0, n0, HALF);
        loads = min(loads, 2);
        for (int c = 0; c < loads; ++c) bx.load(c, &maps.R, n0 + c * cols, row0);
      }
      ok = mbar_wait_cluster(&tmem_full[acc], acc_phase, wd);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
      auto part_row0 = [&](int w) { return (w * 2 + static_cast<int>(rank)) * BM + quarter * 32; };
      if (seg.role == kSegPartial) {
        for (int i = 0; i < PARTS; ++i)
          epilogue_tma<PART_COLS, GEMM_F32>(&maps.P, t_row + part_col(i), bx.mem, bx.next, lane,
                                            part_row0(cluster_id), part_col(i), INT32_MAX, BN);
        if (lane == 0) {
          bulk_wait_group<0>();
          fence_proxy_async_global();
          st_release_gpu(p.sk_flags + (cluster_id * 2 + rank) * kPairEpiWarps + e, epoch);
        }
        __syncwarp();
      } else {
        if (seg.role == kSegOwner) {
          // The workers first_src..last_src computed the start of this tile: add their
          // partials in order. The owner piece is its worker's last, so the ring is idle and
          // each warp borrows a slice of it for the partial's rows.
          uint8_t *slice = smem + e * PART_BYTES;
          for (int w = seg.first_src; ok && w <= seg.last_src; ++w) {
            ok = wait_flag(p.sk_flags + (w * 2 + rank) * kPairEpiWarps + e, epoch, wd);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_proxy_async_global();
            if (w != seg.first_src) {
              __syncwarp();               // every lane has read the previous partial
              fence_proxy_async_smem();   // before the TMA unit writes over it
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(&part_bar[e], PART_BYTES);
#pragma unroll
              for (int c = 0; c < HALF / 32; ++c)
                tma_load_2d(smem_u32(slice + c * kStoreBufBytes), &maps.P, smem_u32(&part_bar[e]),
                            part_col(c * 32 / PART_COLS) + c * 32 % PART_COLS, part_row0(w));
            }
            ok = mbar_wait(&part_bar[e], part_phase, wd);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
              if (lane == 0) drain_wait(&part_bar[e], part_phase, p.f.timeout_ns);
              __syncwarp();
              break;
            }
            part_phase ^= 1;
            for (int i = 0; i < PARTS; ++i)
              add_partial_into_tmem<PART_COLS>(t_row + part_col(i),
                                               slice + i * (PART_BYTES / PARTS), lane);
          }
          if (!ok) break;
        }
        const uint32_t t_cols = t_row + out_half;  // g's columns in the gated accumulator
        if (p.tma_out) {
          if (GATED) {
            if (p.f.out_dtype == GEMM_BF16)
              gated_boxes<GEMM_BF16>(maps, p, bx, t_cols, row0, n0);
            else
              gated_boxes<GEMM_F16>(maps, p, bx, t_cols, row0, n0);
          } else if (p.f.out_dtype == GEMM_BF16) {
            ok = plain_boxes<GEMM_BF16>(maps, p, bx, t_cols, row0, n0, wd);
          } else if (p.f.out_dtype == GEMM_F16) {
            ok = plain_boxes<GEMM_F16>(maps, p, bx, t_cols, row0, n0, wd);
          } else {
            ok = plain_boxes<GEMM_F32>(maps, p, bx, t_cols, row0, n0, wd);
          }
          if (!ok) break;
        } else if (p.f.out_dtype == GEMM_BF16) {
          direct_rows<__nv_bfloat16, GATED>(p, t_cols, row0 + lane, n0);
        } else if (p.f.out_dtype == GEMM_F16) {
          direct_rows<__half, GATED>(p, t_cols, row0 + lane, n0);
        } else if (!GATED) {
          direct_rows<float, GATED>(p, t_cols, row0 + lane, n0);
        }
      }
      loads = 0;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (lane == 0) {
      // after an abort, residual loads may still be landing in the boxes (their barriers'
      // parities are those of the loads not yet waited for)
      if (loads)
        for (int b = 0; b < 2; ++b) drain_wait(&bx.bars[b], (bx.phases >> b) & 1u, p.f.timeout_ns);
      bulk_wait_group<0>();
    }
    __syncwarp();
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&xs[3])), rank ^ 1u),
                          *abort_flag ? 1u : 0u);
    if (!leader) st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&xs[2])), 0), xs[0]);
  }
  tc_fence_before();
  cluster_sync();
  if (*abort_flag || xs[3]) {
    if (leader && threadIdx.x == 0)
      drain_pair_fills<STAGES>(full, xs[1], xs[0], xs[2], STAGE_BYTES, p.f.timeout_ns);
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * BN);
  }
  if (split && threadIdx.x == 0) sk_epoch_end(p.sk_epoch_word, epoch);
}

template <bool GATED, bool W_MN>
cudaError_t launch_pair(const PairMaps &maps, const PairParams &p, int grid, cudaStream_t s) {
  auto kernel = pair_kernel<GATED, W_MN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
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
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

}  // namespace

cudaError_t pair_launch(bool gated, bool w_mn, const PairMaps &maps, const PairParams &p, int grid,
                        cudaStream_t s) {
  if (gated)
    return w_mn ? launch_pair<true, true>(maps, p, grid, s) : launch_pair<true, false>(maps, p, grid, s);
  return w_mn ? launch_pair<false, true>(maps, p, grid, s) : launch_pair<false, false>(maps, p, grid, s);
}

}  // namespace ff
}  // namespace gemm_gb300
