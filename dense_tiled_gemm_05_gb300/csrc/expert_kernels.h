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
  int32_t panels;          // w_mn: a stage's weights come in one copy
  int32_t up_first;        // interleaved pair: the up projection's 16 rows come before the gate's
  void *C;
  int64_t ldc;
  void *pre, *pre2;        // gated: receive the two products, or null
  int64_t ld_pre, ld_pre2;
  int32_t wide;            // all rows stored start on 8-byte boundaries, and N is a multiple of four
  // sums of split tiles: [cluster][CTA][column][128], flags and epoch as in TcParams
  // (stream_k: GEMM_OPT_STREAM_K)
  int32_t stream_k;
  float *sk_partials;
  int *sk_flags;
  int *sk_epoch_word;
  int *status;
  uint64_t timeout_ns;
  int32_t debug_flags;
};
// X, X2: {K, rows} in boxes of 64 x 32, 64, 96 and 128. W, W2: {K, N, experts} in boxes of 64 x 128, or
// (w_mn) {64, K, N / 64, experts} in boxes of 64 x 64 x 2 where N allows it (p.panels), else
// {N, K, experts} in boxes of 64 x 64; an interleaved pair {K, 16, 2, N / 16, experts} in boxes of
// 64 x 16 x 2 x 4, the third axis leading from one matrix to the other.
struct ExpertMaps {
  CUtensorMap X[4], X2[4], W, W2;
};
// How a call runs: one product; a gated pair whose weights come interleaved, 16 rows of each in
// turn (K-contiguous weights); or a gated pair in two accumulators.
enum ExpertMode { kExpertPlain, kExpertMixed, kExpertTwo };
__host__ __device__ constexpr int expert_features(int mode) { return mode == kExpertMixed ? 128 : 256; }
__host__ __device__ constexpr int expert_tokens(int mode, bool narrow) {
  return narrow ? 64 : mode == kExpertTwo ? 128 : 256;
}
// narrow: for few rows an expert (not with kExpertTwo).
cudaError_t expert_launch(ExpertMode mode, bool w_mn, bool narrow, const ExpertMaps &maps,
                          const ExpertParams &p, int grid, cudaStream_t s);
// Clusters of two CTAs of these kernels, one an SM, that fit on the current device at once.
int expert_max_clusters();
// Floats of a cluster's sums of split tiles.
inline int64_t expert_share_floats(bool narrow) { return 2 * 128 * (narrow ? 64 : 256); }

// D[e] = sum over the rows r of expert e of A[r]^T B[r].
struct ExpertGradParams {
  const int32_t *offsets;
  int32_t experts, rows;
  int32_t MA, NB;          // D's rows and columns
  int32_t tiles_m, tiles_n;
  uint32_t idesc;
  int32_t dtype;
  int32_t tma_out;         // D is TMA-addressable
  int32_t panels_a, panels_b;  // a stage's operand comes in one copy
  void *D;
  int64_t ldd, stride_d;
  int *status;
  uint64_t timeout_ns;
  int32_t debug_flags;
};
// A: {64, rows, MA / 64} in boxes of 64 x 64 x 2 where MA allows it (panels_a), else {MA, rows} in
// boxes of 64 x 64; B likewise; D: {NB, MA, experts} in boxes of 64 x 32.
struct ExpertGradMaps {
  CUtensorMap A, B, D;
};
cudaError_t expert_grad_launch(const ExpertGradMaps &maps, const ExpertGradParams &p, int grid,
                               cudaStream_t s);

// fp32: C[r] (+)= A[r] B[e] for the rows of each expert (A: rows x K, B: K x N each), or, with grad,
// C[e] = sum over e's rows of A[r]^T B[r] (M x N each). Element (i, k) of an operand is at
// i * line + k * step, i being C's row or column and k the summed index; line or step is 1.
struct ExpertF32Params {
  const int32_t *offsets;
  int32_t experts, rows;
  int32_t M, N;            // M: grad only
  int64_t K;               // not grad
  const float *A, *B;
  int64_t a_line, a_step, b_line, b_step;
  int64_t stride_b;        // from expert to expert (not grad)
  float *C;
  int64_t ldc, stride_c;   // stride_c: grad only
  int32_t add;
};
cudaError_t expert_f32_launch(bool grad, const ExpertF32Params &p, int sm_count, cudaStream_t s);

}  // namespace ff
}  // namespace gemm_gb300
