// ff_kernels.h -- parameters and launchers of the feed-forward operators' tensor-core
// kernels: products of 16-bit operands with an epilogue, and the gated pair.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ff_internal.h"
#include "internal.h"

namespace gemm_gb300 {
namespace ff {

// What both kernels compute. Plain: C = act(X W + bias) + residual, where the product may be
// the sum of two (X W + X2 W2: the K-blocks from kb_first on come from the second pair).
// Gated: C = act(X W) * (X W2), `pre` and `pre2` receiving the two products.
struct FusedParams {
  int32_t M, N;         // tokens, output features
  int32_t k_blocks;     // 64-long K-blocks
  int32_t kb_first;     // those of the first pair (k_blocks when there is one)
  uint32_t idesc;       // tcgen05 instruction descriptor
  int32_t out_dtype;
  int32_t act;
  int32_t bias_dtype;
  const void *bias;
  const void *residual;
  int64_t ld_residual;
  void *C;
  int64_t ldc;
  void *pre;
  int64_t ld_pre;
  void *pre2;           // gated only
  int64_t ld_pre2;
  int *status;
  uint64_t timeout_ns;
  int32_t debug_flags;
};

// Few-token kernel: features on the MMA's M side, tokens on its N side.
struct FewParams {
  FusedParams f;
  int32_t tile_t;       // tokens per tile: a multiple of 16, at most 256 (gated: 128)
  int32_t tiles_t, tiles_f;
  int32_t splits;       // CTAs (one cluster) that share a tile's K-blocks: 1, 2, 4 or 8
  int32_t stages;       // ring stages
  int32_t vec;          // outputs, residual and bias allow 4-element accesses
};
constexpr int kFewFeatures = 128;  // features per tile
constexpr size_t kFewFixedBytes = 2048;  // barriers and alignment (at most)
size_t few_stage_bytes(bool gated, int tile_t);
size_t few_smem_bytes(bool gated, int tile_t, int stages, bool split);
// Clusters of `splits` CTAs, one an SM, that run at once on the current device.
int few_max_clusters(int splits);
cudaError_t few_launch(bool gated, bool w_mn, const CUtensorMap &tmX, const CUtensorMap &tmW,
                       const CUtensorMap &tmX2, const CUtensorMap &tmW2, const FewParams &p,
                       cudaStream_t s);

// Token kernel: one to eight tokens against K-contiguous weights of any alignment, on fp32
// fused multiply-adds.
struct TokenParams {
  FusedParams f;        // (k_blocks, kb_first and idesc unused)
  const void *X;
  int64_t ldx;
  const void *W, *W2;   // W2: gated only
  int64_t ldw, ldw2;
  int64_t K;
  int32_t k_warps;      // warps of a CTA that share a feature's K: 1, 2, 4 or 8
};
constexpr int kTokenMax = 8;
// vector: X and weights allow 16-byte accesses and K is a multiple of them.
cudaError_t token_launch(bool gated, int dtype, bool vector, const TokenParams &p, cudaStream_t s);

// fp32 tile kernel: exact products on fused multiply-adds, operands of any layout and
// alignment. X is M x K, W is K x N; *_k: K is the contiguous axis.
struct TileParams {
  FusedParams f;        // (k_blocks, kb_first and idesc unused)
  const float *X, *W, *W2;
  int64_t ldx, ldw, ldw2;
  int32_t x_k, w_k;
  int64_t K;
  int32_t splits;       // CTAs (one cluster) that share a tile's K: 1, 2, 4 or 8
  int32_t run_steps;    // K-steps an accumulator adds up before its sum moves on (tile_run_steps)
  int32_t vec;          // as FewParams
};
constexpr int kTileK = 16;  // K elements per step
// Rows and columns of a tile (gated: columns of each product) for a size of 64 or 128.
inline int tile_rows(int size) { return size; }
inline int tile_cols(bool gated, int size) { return gated ? size / 2 : size; }
int tile_run_steps(int64_t K);
cudaError_t tile_launch(bool gated, int size, const TileParams &p, cudaStream_t s);

// Many-token kernel: CTA pairs, 256 x 256 accumulators (gated: 128 columns of each product).
struct PairParams {
  FusedParams f;
  int32_t tiles_m, tiles_n;
  int32_t group_m;      // tile rows per raster group
  int32_t tma_out;      // outputs and residual are TMA-addressable
  // split-K share of the last rounds, as in TcParams
  int32_t sk_dp_tiles;
  float *sk_partials;
  int *sk_flags;
  int *sk_epoch_word;
};
// Operand maps (first and second pair), outputs, kept products, residual, split-K partials.
struct PairMaps {
  CUtensorMap X, W, X2, W2, C, Z, Z2, R, P;
};
cudaError_t pair_launch(bool gated, bool w_mn, const PairMaps &maps, const PairParams &p, int grid,
                        cudaStream_t s);

}  // namespace ff
}  // namespace gemm_gb300
