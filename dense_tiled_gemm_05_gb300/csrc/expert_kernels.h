// expert_kernels.h -- parameters and launchers of the experts' products: rows sorted by expert,
// each expert's rows against its own weights.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "expert_internal.h"
#include "internal.h"

namespace gemm_gb300 {
namespace ff {

// Y[r] = X[r] W[e] for the rows r of each expert e, or the sum of two products (the K-blocks from
// kb_first on come from X2 and W2), or (gated) act(X W) * (X W2).
struct ExpertParams {
  const int32_t *offsets;  // experts + 1
  int32_t experts, rows;
  int32_t N;               // output features
  int32_t k_blocks;        // 64-long K-blocks
  int32_t kb_first;        // those of the first pair
  uint32_t idesc;          // tcgen05 instruction descriptor without its N
  int32_t dtype, act;
  void *C;
  int64_t ldc;
  void *pre, *pre2;        // gated: receive the two products, or null
  int64_t ld_pre, ld_pre2;
  int *status;
  uint64_t timeout_ns;
  int32_t debug_flags;
};
// X, X2: {K, rows} in boxes of 64 x 32. W, W2: {K, N, experts} in boxes of 64 x 128 or (w_mn)
// {N, K, experts} in boxes of 64 x 64.
struct ExpertMaps {
  CUtensorMap X, X2, W, W2;
};
constexpr int kExpertFeatures = 256;  // features a tile
inline int expert_tile_tokens(bool gated) { return gated ? 128 : 256; }  // tokens a tile, at most
cudaError_t expert_launch(bool gated, bool w_mn, const ExpertMaps &maps, const ExpertParams &p,
                          int grid, cudaStream_t s);
// Clusters of two CTAs of these kernels that fit on the current device at once.
int expert_max_clusters();

// D[e] = sum over the rows r of expert e of A[r]^T B[r].
struct ExpertGradParams {
  const int32_t *offsets;
  int32_t experts, rows;
  int32_t MA, NB;          // D's rows and columns
  int32_t tiles_m, tiles_n;
  uint32_t idesc;
  int32_t dtype;
  int32_t tma_out;         // D is TMA-addressable
  void *D;
  int64_t ldd, stride_d;
  int *status;
  uint64_t timeout_ns;
  int32_t debug_flags;
};
// A: {MA, rows}, B: {NB, rows} in boxes of 64 x 64; D: {NB, MA, experts} in boxes of 64 x 32.
struct ExpertGradMaps {
  CUtensorMap A, B, D;
};
cudaError_t expert_grad_launch(const ExpertGradMaps &maps, const ExpertGradParams &p, int grid,
                               cudaStream_t s);

}  // namespace ff
}  // namespace gemm_gb300
