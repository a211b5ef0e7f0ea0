// ff_tile_kernel.cu -- small exact fp32 products with an epilogue, and the gated pair, on fp32
// fused multiply-adds:
//
//   Y = act(X W + bias) + residual      or      H = act(X Wg) * (X Wu)
//
// The exact product on the tensor cores (tf32 parts, partial sums drained every chunk) has at
// least 30 us of splitting and chunk drains whatever its size; below about 2.5 GFLOP plain
// multiply-adds are done sooner. A CTA computes a 128 x 128 or 64 x 64 tile, 8 x 8 or 8 x 4
// outputs a thread (gated: half the columns of each product), so that a K-step takes 64 or 32
// multiply-adds for four or three 16-byte shared-memory reads. Operands arrive by 4-byte
// cp.async -- any alignment, the ragged edges filled with zeros -- and are laid down K-major,
// transposed on the way where K is their contiguous axis, in a ring of three 16-long steps.
// At 128 registers an SM holds 16 warps, which leave half of the issue slots unused (0.45 issued
// a cycle and scheduler on 1023 x 1025 x 1000: 60.4 us, 35 TFLOP/s, one GB300; 42 on 3000 x 1000
// x 2000, cuBLAS 51).
// Where tiles are few, a cluster's CTAs share each tile's K and join as in ff_join.cuh.
//
// A share of K is added up in runs (tile_run_steps), whose sums are added in shared memory: a sum
// of n terms of one sign in a row loses about sqrt(n) roundings of its own size (n = 8192 in each
// of eight shares: 2e-6 of sum |x w|, twice the bound of exact products; in runs 6e-7). On
// one GB300 that takes 2 % of 1023 x 1025 x 1000 and 7 % of 64 x 2048 x 8192.
#include <cmath>

#include "ff_join.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

// One thread's share of the loads of a ROWS x 16 operand tile into smem[k][row], zero outside
// the operand. k_inner: element (r, k) is at p[r * ld + k], and the threads of a tile's row
// take its K; else at p[k * ld + r], and they take neighbouring rows. A thread's elements
// are `turn` apart, so that a copy costs an address addition.
template <int ROWS, int THREADS>
struct Loader {
  static constexpr int N = ROWS * kTileK / THREADS;
  const float *src;    // its first element of the current step
  int64_t turn, step;  // between its elements, and between steps
  uint32_t in;         // bit i: element i's row is in the operand
  int k, k_turn;       // K of its first element in the step, and between elements
  int dst, dst_turn;   // offsets in the tile
  __device__ __forceinline__ Loader(const float *p, int64_t ld, bool k_inner, int64_t r0,
                                    int64_t rows, int64_t k0) {
    const int t = threadIdx.x;
    // k_inner: a warp takes 8 K of 4 rows -- whole 32-byte sectors of the operand and, rows of
    // the tile being 4 banks apart, all 32 banks
    const int r = k_inner ? t / 64 * 4 + t / 8 % 4 : t % ROWS;
    const int r_turn = k_inner ? THREADS / kTileK : 0;
    k = k_inner ? t / 32 % 2 * 8 + t % 8 : t / ROWS;
    k_turn = k_inner ? 0 : THREADS / ROWS;
    in = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) in |= (r0 + r + i * r_turn < rows ? 1u : 0u) << i;
    src = p + (k_inner ? (r0 + r) * ld + k0 + k : (k0 + k) * ld + r0 + r);
    turn = k_inner ? r_turn * ld : k_turn * ld;
    step = k_inner ? kTileK : kTileK * ld;
    dst = k * (ROWS + 4) + r;
    dst_turn = k_turn * (ROWS + 4) + r_turn;
  }
  // k_left: K elements from this step on.
  __device__ __forceinline__ void load(float *tile, int64_t k_left) {
    const uint32_t to = smem_u32(tile + dst);
    if (in == (1u << N) - 1u && k_left >= kTileK) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + i * dst_turn * 4),
                     "l"(src + i * turn)
                     : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if ((in >> i & 1u) && k + i * k_turn < k_left)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + i * dst_turn * 4),
                       "l"(src + i * turn)
                       : "memory");
        else
          tile[dst + i * dst_turn] = 0.0f;
      }
    }
    src += step;
  }
};
static_assert(kTileK == 16, "the K of two warps");

// RUNS: shares of K of several runs.
template <int BM_, int BN_, int TM_, int TN_, bool GATED, bool RUNS_>
struct Tile {
  static constexpr int S = GATED ? 2 : 1;
  static constexpr bool RUNS = RUNS_;
  // (the sums of a 128 x 128 tile leave room for two stages where two CTAs share an SM)
  static constexpr int STAGES = RUNS && BM_ == 128 ? 2 : 3;
  static constexpr int BM = BM_, BN = BN_, TM = TM_, TN = TN_;
  static constexpr int TX = BN / TN, TY = BM / TM, THREADS = TX * TY;
  struct Stage {
    float x[kTileK][BM + 4];
    float w[S][kTileK][BN + 4];
  };
  static constexpr int RING = STAGES * static_cast<int>(sizeof(Stage));
  static constexpr int PART = S * BM * BN * 4;
  // the partial lies over the ring, or behind it where runs are added up there
  static constexpr int SMEM = RUNS ? RING + PART : RING > PART ? RING : PART;
  static_assert(BM * kTileK % THREADS == 0 && BN * kTileK % THREADS == 0 && THREADS % BM == 0 &&
                    THREADS % BN == 0 && TM % 4 == 0 && TN % 4 == 0,
                "whole shares");
};

__device__ __forceinline__ void read4(const float *p, float *v) {
  const float4 q = *reinterpret_cast<const float4 *>(p);
  v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(T::THREADS, 512 / T::THREADS)
    tile_kernel(const TileParams p) {
  constexpr int S = T::S, BM = T::BM, BN = T::BN, TM = T::TM, TN = T::TN, THREADS = T::THREADS;
  constexpr int STAGES = T::STAGES;
  extern __shared__ __align__(16) uint8_t dyn[];
  typename T::Stage *ring = reinterpret_cast<typename T::Stage *>(dyn);
  const int rank = static_cast<int>(blockIdx.x) % p.splits;
  const int64_t tile = blockIdx.x / p.splits;
  const int64_t tiles_m = (p.f.M + BM - 1) / BM;
  const int64_t m0 = tile % tiles_m * BM, n0 = tile / tiles_m * BN;
  const int64_t steps = (p.K + kTileK - 1) / kTileK;
  const int lo = static_cast<int>(steps * rank / p.splits);
  const int n_steps = static_cast<int>(steps * (rank + 1) / p.splits) - lo;
  const int64_t k0 = int64_t{lo} * kTileK;
  // a thread's rows (columns) are groups of four, TY (TX) threads' groups apart
  const int tx = threadIdx.x % T::TX, ty = threadIdx.x / T::TX;
  Loader<BM, THREADS> lx(p.X, p.ldx, p.x_k, m0, p.f.M, k0);
  Loader<BN, THREADS> lw(p.W, p.ldw, p.w_k, n0, p.f.N, k0);
  Loader<BN, THREADS> lw2(GATED ? p.W2 : p.W, GATED ? p.ldw2 : p.ldw, p.w_k, n0, p.f.N, k0);
  grid_dependency_wait();
  grid_launch_dependents();
  auto fetch = [&](int step) {
    if (step < n_steps) {
      typename T::Stage &g = ring[step % STAGES];
      const int64_t left = p.K - k0 - int64_t{step} * kTileK;
      lx.load(&g.x[0][0], left);
      lw.load(&g.w[0][0][0], left);
      if (GATED) lw2.load(&g.w[S - 1][0][0], left);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  F2 acc[S][TM / 2][TN];  // pairs of rows: two multiply-adds an instruction
  // The partial, [row][column], over the drained ring or (RUNS) behind it: the accumulators
  // replace it or, after the first run, are added to it. A thread's elements are its own.
  float *part = reinterpret_cast<float *>(dyn + (T::RUNS ? T::RING : 0));
  bool begun = false;
  int run_left = p.run_steps;
  auto to_partial = [&] {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < TM; i += 2) {
        const int r = i / 4 * 4 * T::TY + ty * 4 + i % 4;
#pragma unroll
        for (int j = 0; j < TN; j += 4) {
          float2 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = acc[s][i / 2][j + c].get();
          float *d = part + s * BM * BN + r * BN + j * T::TX + tx * 4;
          float4 lo = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
          float4 hi = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
          if (T::RUNS && begun) {
            const float4 a = *reinterpret_cast<const float4 *>(d);
            const float4 b = *reinterpret_cast<const float4 *>(d + BN);
            lo.x += a.x, lo.y += a.y, lo.z += a.z, lo.w += a.w;
            hi.x += b.x, hi.y += b.y, hi.z += b.z, hi.w += b.w;
          }
          *reinterpret_cast<float4 *>(d) = lo;
          *reinterpret_cast<float4 *>(d + BN) = hi;
        }
      }
    begun = true;
  };
  for (int k = 0; k < STAGES - 1; ++k) fetch(k);
  for (int step = 0; step < n_steps; ++step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncthreads();  // the step's tiles are there; everyone is done with the stage refilled next
    fetch(step + STAGES - 1);
    const typename T::Stage &g = ring[step % STAGES];
#pragma unroll
    for (int k = 0; k < kTileK; ++k) {
      float a[TM];
#pragma unroll
      for (int i = 0; i < TM; i += 4) read4(&g.x[k][i * T::TY + ty * 4], &a[i]);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float b[TN];
#pragma unroll
        for (int j = 0; j < TN; j += 4) read4(&g.w[s][k][j * T::TX + tx * 4], &b[j]);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const F2 bb(b[j], b[j]);
#pragma unroll
          for (int i = 0; i < TM / 2; ++i)
            acc[s][i][j] = fma2(F2(a[2 * i], a[2 * i + 1]), bb, acc[s][i][j]);
        }
      }
    }
    if (T::RUNS && --run_left == 0 && step + 1 < n_steps) {
      run_left = p.run_steps;
      to_partial();
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < TM / 2; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[s][i][j] = F2();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring is free
  to_partial();  // also of a tile computed alone, so that the stores that follow are whole rows
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  const int rows = static_cast<int>(p.f.M - m0 < BM ? p.f.M - m0 : BM);
  join_partials<GATED, false, BN, THREADS, 4>(p.f, p.vec, smem_u32(part), BM * BN, rows, p.splits,
                                              rank, m0, n0);
  if (p.splits > 1) cluster_sync();  // the other CTAs may still be reading this one's partial
}

template <typename T, bool GATED>
cudaError_t launch_tile(const TileParams &p, cudaStream_t s) {
  auto kernel = tile_kernel<T, GATED>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.f.M + T::BM - 1) / T::BM) * ((p.f.N + T::BN - 1) / T::BN);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dependency_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.splits), 1, 1);
  cfg.blockDim = dim3(T::THREADS, 1, 1);
  cfg.dynamicSmemBytes = T::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool GATED, bool RUNS>
cudaError_t dispatch(int size, const TileParams &p, cudaStream_t s) {
  if (size == 128) return launch_tile<Tile<128, GATED ? 64 : 128, 8, GATED ? 4 : 8, GATED, RUNS>, GATED>(p, s);
  if (size == 64) return launch_tile<Tile<64, GATED ? 32 : 64, GATED ? 4 : 8, 4, GATED, RUNS>, GATED>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace

// Steps an accumulator adds up in a row: at least 128 products, or 8 sqrt(K). The K / r runs of
// r products are summed in order, and their errors, of some sqrt(r) roundings of a run's sum,
// average out to r / sqrt(K) roundings of the whole: 8 of 2^-24, 5e-7.
int tile_run_steps(int64_t K) {
  const double r = 8.0 * std::sqrt(static_cast<double>(K));
  return static_cast<int>(r < 128.0 ? 128.0 : r) / kTileK;
}

cudaError_t tile_launch(bool gated, int size, const TileParams &p, cudaStream_t s) {
  const int64_t steps = (p.K + kTileK - 1) / kTileK;
  const bool runs = (steps + p.splits - 1) / p.splits > p.run_steps;
  if (p.run_steps < 1) return cudaErrorInvalidValue;
  if (gated) return runs ? dispatch<true, true>(size, p, s) : dispatch<true, false>(size, p, s);
  return runs ? dispatch<false, true>(size, p, s) : dispatch<false, false>(size, p, s);
}

}  // namespace ff
}  // namespace gemm_gb300
