// ff_few_kernel.cu -- products of few tokens with an epilogue, and the gated pair:
//
//   Y = act(X W + bias) + residual      or      H = act(X Wg) * (X Wu)
//
// for X of a few to some hundred rows. Such a product is bound by reading the weights once
// (2 flops per weight and token against ~280 per byte at the ridge), so the layout puts the
// weights where the tensor core is widest: 128 output features are the MMA's M rows and the
// tokens, 16 to 256 of them, its N columns -- one token costs a 16-column MMA instead of a
// 128-row tile of padding. TMA streams 128 x 64 weight boxes through a ring of stages that
// fills shared memory, which keeps enough bytes in flight on every SM for HBM.
//
// A tile's K-loop alone would leave most SMs idle (4096 features are 32 tiles), so a cluster
// of 2, 4 or 8 CTAs shares it: each accumulates its K-blocks in TMEM, writes the fp32 partial
// to its shared memory (over the drained ring), and after a cluster barrier every CTA sums a
// share of the outputs over all partials through distributed shared memory, in rank order,
// applies the epilogue and stores. No workspace, no second launch, the same bits every time. A
// tile that is not split goes from TMEM to memory directly.
//
// The gated pair runs as two MMAs a K-step, both weights' rows against the same token tile.
#include <atomic>

#include "ff_join.cuh"
#include "tc_common.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

using namespace tc;

// Warp 0 loads, warp 1 issues the MMAs, warps 4-11 (two for each quarter of the TMEM lanes)
// read the accumulators; all twelve sum the partials of a split tile.
constexpr int kFewThreads = 384;
constexpr int kBlockK = 64;                          // K elements per 128-byte K-block
constexpr int kWBytes = kFewFeatures * kRowBytes;    // one weight box
constexpr int kPanelBytes = kBlockK * kRowBytes;     // MN-major weights: 64 K-rows x 128 bytes
constexpr int kMaxStages = 16;
constexpr int kBarBytes = (2 * kMaxStages + 2) * 8 + 16;
static_assert(kBarBytes + 1024 <= kFewFixedBytes, "barriers and alignment");

// TMEM columns between the two accumulators of a gated tile, and to allocate.
__host__ __device__ constexpr int acc_stride(int tile_t) {
  return tile_t <= 32 ? 32 : tile_t <= 64 ? 64 : tile_t <= 128 ? 128 : 256;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The box that tma_load_2d takes at the same coordinates, into L2 only.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *m, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y)
               : "memory");
}

// One feature a lane, 16 tokens of its TMEM columns: the epilogue of a tile that one CTA
// computed alone. A warp's 32 features of a token are neighbours in memory.
template <typename TO, bool GATED>
__device__ __forceinline__ void finish_columns(const FusedParams &p, int64_t m0, int tokens, int64_t n,
                                               float bias, float (&a)[16], float (&b)[16]) {
  if (n >= p.N) return;
  if (GATED) {
    if (p.pre) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < tokens) {
          static_cast<TO *>(p.pre)[(m0 + j) * p.ld_pre + n] = from_f32<TO>(a[j]);
          static_cast<TO *>(p.pre2)[(m0 + j) * p.ld_pre2 + n] = from_f32<TO>(b[j]);
        }
    }
    activate_all<true>(a, p.act);
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] *= b[j];
  } else {
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        b[j] = j < tokens ? to_f32(static_cast<const TO *>(p.residual)[(m0 + j) * p.ld_residual + n]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] += bias;
    if (p.pre) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < tokens) static_cast<TO *>(p.pre)[(m0 + j) * p.ld_pre + n] = from_f32<TO>(a[j]);
    }
    activate_all<true>(a, p.act);
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < 16; ++j) a[j] += b[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < tokens) static_cast<TO *>(p.C)[(m0 + j) * p.ldc + n] = from_f32<TO>(a[j]);
}

template <bool GATED, bool W_MN>
__global__ void __launch_bounds__(kFewThreads)
    few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmX2, const __grid_constant__ CUtensorMap tmW2,
               const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int w_bytes = GATED ? 2 * kWBytes : kWBytes;
  const int x_bytes = p.tile_t * kRowBytes;
  const int stage_bytes = w_bytes + x_bytes;
  const int accs = GATED ? 2 : 1;
  const int plane = p.tile_t * kFewFeatures;  // fp32 values of one accumulator's partial
  const int ring = p.stages * stage_bytes;
  const int part = p.splits > 1 ? accs * plane * static_cast<int>(sizeof(float)) : 0;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + (ring > part ? ring : part));
  uint64_t *empty = full + kMaxStages;
  uint64_t *acc_full = empty + kMaxStages;
  uint64_t *drain = acc_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int rank = static_cast<int>(blockIdx.x) % p.splits;  // == rank in the cluster
  const int tile = static_cast<int>(blockIdx.x) / p.splits;
  // token tiles run fastest: the CTAs in flight share weights through L2
  const int t0 = tile % p.tiles_t * p.tile_t, f0 = tile / p.tiles_t * kFewFeatures;
  const int tokens = min(p.tile_t, p.f.M - t0);
  const int kb_lo = static_cast<int>(static_cast<int64_t>(rank) * p.f.k_blocks / p.splits);
  const int kb_hi = static_cast<int>(static_cast<int64_t>(rank + 1) * p.f.k_blocks / p.splits);
  auto in_second = [&](int kb) { return !GATED && kb >= p.f.kb_first; };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t tmem_cols = static_cast<uint32_t>(accs * acc_stride(p.tile_t));
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
    // The ring's first weights are asked into L2 while the previous kernel ends. They are read
    // after the wait, from L2, so that weights which that kernel writes are seen as written.
    // (64 x 4096 x 4096 bf16, calls one after another: 13.8 us without, 13.0 with; 64 x 8192 x
    // 2048: 12.6 and 12.8.)
    for (int kb = kb_lo; kb < min(kb_lo + p.stages, kb_hi); ++kb) {
      const bool second = in_second(kb);
      const int k0 = (second ? kb - p.f.kb_first : kb) * kBlockK;
#pragma unroll
      for (int i = 0; i < (GATED ? 2 : 1); ++i) {
        const CUtensorMap *m = (GATED ? i == 1 : second) ? &tmW2 : &tmW;
        if (W_MN) {
          tma_prefetch_2d(m, f0, k0);
          tma_prefetch_2d(m, f0 + kBlockK, k0);
        } else {
          tma_prefetch_2d(m, k0, f0);
        }
      }
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // The prologue above may overlap the previous kernel on the stream; global memory is read
  // and written only from here on.
  grid_dependency_wait();
  grid_launch_dependents();
  const Watchdog wd{abort_flag, p.f.status, p.f.timeout_ns};

  uint32_t issued = 0;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      const bool stall = (p.f.debug_flags & kDebugStallProducer) != 0;
      const int stop_after = stall_after_fills(p.f.debug_flags & ~kDebugStallRank1, 0);
      const uint64_t keep = l2_policy_evict_last();
      for (int kb = kb_lo; kb < kb_hi && !stall; ++kb) {
        if (stop_after >= 0 && issued >= static_cast<uint32_t>(stop_after)) break;  // test hook
        if (!mbar_wait(&empty[stage], phase ^ 1, wd)) break;
        mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(stage_bytes));
        const uint32_t w_dst = smem_u32(smem + stage * stage_bytes);
        const uint32_t fb = smem_u32(&full[stage]);
        const bool second = in_second(kb);
        const int k0 = (second ? kb - p.f.kb_first : kb) * kBlockK;
#pragma unroll
        for (int i = 0; i < (GATED ? 2 : 1); ++i) {
          const CUtensorMap *m = (GATED ? i == 1 : second) ? &tmW2 : &tmW;
          const uint32_t dst = w_dst + i * kWBytes;
          if (W_MN) {
            tma_load_2d(dst, m, fb, f0, k0);
            tma_load_2d(dst + kPanelBytes, m, fb, f0 + kBlockK, k0);
          } else {
            tma_load_2d(dst, m, fb, k0, f0);
          }
        }
        tma_load_2d_hint(w_dst + w_bytes, second ? &tmX2 : &tmX, fb, k0, t0, keep);
        ++issued;
        if (++stage == static_cast<uint32_t>(p.stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!mbar_wait(&full[stage], phase, wd)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w_base = smem_u32(smem + stage * stage_bytes);
        const uint32_t x_base = w_base + w_bytes;
#pragma unroll
        for (int kk = 0; kk < kBlockK / 16; ++kk) {
          const uint64_t xd = sdesc_sw128(x_base + kk * 32, 16, 1024);
          const uint32_t accumulate = kb != kb_lo || kk != 0;
#pragma unroll
          for (int i = 0; i < (GATED ? 2 : 1); ++i) {
            const uint32_t w = w_base + i * kWBytes;
            const uint64_t ad = W_MN ? sdesc_sw128(w + kk * 16 * kRowBytes, kPanelBytes, 1024)
                                     : sdesc_sw128(w + kk * 32, 16, 1024);
            mma_f16(tmem_base + i * acc_stride(p.tile_t), ad, xd, p.f.idesc, accumulate);
          }
        }
        mma_commit(&empty[stage]);
        if (++stage == static_cast<uint32_t>(p.stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) mma_commit(acc_full);
      mma_commit(drain);  // every MMA issued above completes before TMEM is released
      drain_wait(drain, 0, p.f.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------- accumulators: to the outputs, or to shared memory
    const int quarter = warp & 3, half = (warp - 4) / 4;
    const int64_t n = f0 + quarter * 32 + lane;
    if (p.splits > 1 && warp == 4 && rank == 0 && !GATED) {
      // what the epilogue reads besides the sums is on its way to L2 meanwhile
      const int es = p.f.out_dtype == GEMM_F32 ? 4 : 2;
      const int cols = min(kFewFeatures, p.f.N - f0);
      if (p.f.bias && lane * 4 < cols)
        prefetch_l2(static_cast<const char *>(p.f.bias) +
                    static_cast<int64_t>(f0 + lane * 4) * (p.f.bias_dtype == GEMM_F32 ? 4 : 2));
      if (p.f.residual)
        for (int t = 0; t < tokens; ++t)
          if (lane * 4 < cols)
            prefetch_l2(static_cast<const char *>(p.f.residual) +
                        ((t0 + t) * p.f.ld_residual + f0 + lane * 4) * es);
    }
    const float bias = !GATED && p.splits == 1 && p.f.bias && n < p.f.N
                           ? load_any(p.f.bias, p.f.bias_dtype, n)
                           : 0.0f;
    bool ok = mbar_wait(acc_full, 0, wd);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      // (the ring is drained: every stage was loaded and read before this barrier completed)
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      float *P = reinterpret_cast<float *>(smem) + quarter * 32 + lane;
      for (int c0 = half * 16; c0 < tokens; c0 += 32) {
        __syncwarp();  // (lanes past N finish early; TMEM is read by whole warps)
        uint32_t r[2][16];
        tmem_ld_32x32b_x16(t_row + c0, r[0]);
        if (GATED) tmem_ld_32x32b_x16(t_row + acc_stride(p.tile_t) + c0, r[1]);
        tmem_wait_ld();
        if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < (GATED ? 2 : 1); ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + j < tokens) P[i * plane + (c0 + j) * kFewFeatures] = __uint_as_float(r[i][j]);
        } else {
          float a[16], b[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            a[j] = __uint_as_float(r[0][j]);
            b[j] = GATED ? __uint_as_float(r[1][j]) : 0.0f;
          }
          const int left = tokens - c0;
          if (p.f.out_dtype == GEMM_BF16)
            finish_columns<__nv_bfloat16, GATED>(p.f, t0 + c0, left, n, bias, a, b);
          else if (p.f.out_dtype == GEMM_F16)
            finish_columns<__half, GATED>(p.f, t0 + c0, left, n, bias, a, b);
          else
            finish_columns<float, GATED>(p.f, t0 + c0, left, n, bias, a, b);
        }
      }
      tc_fence_before();
    }
  }

  // Every partial of a split tile is in its CTA's shared memory after this.
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  if (p.splits > 1)
    join_partials<GATED, true, kFewFeatures, kFewThreads, GATED ? 3 : 6>(
        p.f, p.vec, smem_u32(smem), plane, tokens, p.splits, rank, t0, f0);
  if (threadIdx.x == 0 && *abort_flag) {
    // After an abort, let every copy already issued land: the last fill of stage s is fill
    // number f (f % stages == s), completing parity (f / stages) & 1.
    const uint32_t S = static_cast<uint32_t>(p.stages);
    for (uint32_t s = 0; s < S && s < issued; ++s) {
      const uint32_t f = s + S * ((issued - 1 - s) / S);
      drain_wait(&full[s], (f / S) & 1, p.f.timeout_ns);
    }
  }
  // The other CTAs may still be reading this one's partials.
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

template <bool GATED, bool W_MN>
cudaError_t launch_few(const CUtensorMap &tmX, const CUtensorMap &tmW, const CUtensorMap &tmX2,
                       const CUtensorMap &tmW2, const FewParams &p, cudaStream_t s) {
  auto kernel = few_kernel<GATED, W_MN>;
  const size_t smem = few_smem_bytes(GATED, p.tile_t, p.stages, p.splits > 1);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dependency_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles_t * p.tiles_f * p.splits), 1, 1);
  cfg.blockDim = dim3(kFewThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, tmX, tmW, tmX2, tmW2, p);
}

}  // namespace

// The limit comes from how many SMs each GPC has: one kernel, at one CTA an SM, stands for all.
int few_max_clusters(int splits) {
  static std::atomic<int> cached[64][4];  // per device; 0 = not queried yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 1;
  }
  std::atomic<int> &known = cached[dev][splits == 1 ? 0 : splits == 2 ? 1 : splits == 4 ? 2 : 3];
  const int n = known.load(std::memory_order_relaxed);
  if (n > 0) return n;
  auto kernel = few_kernel<false, false>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(splits), 1, 1);
  cfg.blockDim = dim3(kFewThreads, 1, 1);
  cfg.dynamicSmemBytes = 226 * 1024;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int got = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&got, kernel, &cfg) != cudaSuccess || got < 1) {
    cudaGetLastError();
    return 1;
  }
  known.store(got, std::memory_order_relaxed);
  return got;
}

size_t few_stage_bytes(bool gated, int tile_t) {
  return static_cast<size_t>((gated ? 2 : 1) * kWBytes + tile_t * kRowBytes);
}

// The request is never below a CTA's TMEM columns' share of the SM's 228 KB (456 bytes a
// column, 1 KB a CTA being the system's): CTAs whose shared memory fits an SM together then
// also find their TMEM there, whichever kernels they belong to, and no cluster ever waits for
// columns that another waiting cluster holds.
size_t few_smem_bytes(bool gated, int tile_t, int stages, bool split) {
  const size_t ring = static_cast<size_t>(stages) * few_stage_bytes(gated, tile_t);
  const size_t part = split ? static_cast<size_t>(gated ? 2 : 1) * tile_t * kFewFeatures * sizeof(float) : 0;
  const size_t use = (ring > part ? ring : part) + kBarBytes + 1024;
  const size_t least = static_cast<size_t>((gated ? 2 : 1) * acc_stride(tile_t)) * 456 - 1024;
  return use > least ? use : least;
}

cudaError_t few_launch(bool gated, bool w_mn, const CUtensorMap &tmX, const CUtensorMap &tmW,
                       const CUtensorMap &tmX2, const CUtensorMap &tmW2, const FewParams &p,
                       cudaStream_t s) {
  if (p.stages < 1 || p.stages > kMaxStages || p.tile_t % 16 || p.tile_t < 16 ||
      p.tile_t > (gated ? 128 : 256) || few_smem_bytes(gated, p.tile_t, p.stages, p.splits > 1) > 232448)
    return cudaErrorInvalidValue;
  if (gated)
    return w_mn ? launch_few<true, true>(tmX, tmW, tmX2, tmW2, p, s)
                : launch_few<true, false>(tmX, tmW, tmX2, tmW2, p, s);
  return w_mn ? launch_few<false, true>(tmX, tmW, tmX2, tmW2, p, s)
              : launch_few<false, false>(tmX, tmW, tmX2, tmW2, p, s);
}

}  // namespace ff
}  // namespace gemm_gb300
