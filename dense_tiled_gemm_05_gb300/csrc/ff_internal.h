// ff_internal.h -- launchers of the feed-forward operators' kernels, shared by the C ABI
// (feed_forward.cu) and the kernels' translation units. Internal to the
// library.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace gemm_gb300 {
namespace ff {

// What follows a product in the same call: y = act(z) + residual, z = acc + bias.
struct Epilogue {
  const void *bias = nullptr;  // N values
  int bias_dtype = GEMM_F32;
  int act = GEMM_ACT_NONE;
  const void *residual = nullptr;  // M x N, C's type
  int64_t ld_residual = 0;
  void *pre = nullptr;  // M x N, C's type: z
  int64_t ld_pre = 0;
  bool empty() const { return !bias && act == GEMM_ACT_NONE && !residual && !pre; }
};

// y = act(z + bias) + residual from the fp32 product z (M x N, ldz); y may be z's own buffer.
cudaError_t epilogue_rows_launch(const float *z, int64_t ldz, void *y, int64_t ldy, int out_dtype,
                                 const Epilogue &ep, int64_t M, int64_t N, cudaStream_t s);

// h = act(g) * u from fp32 g and u (M x F).
cudaError_t gated_rows_launch(const float *g, int64_t ldg, const float *u, int64_t ldu, void *h,
                              int64_t ldh, int out_dtype, int act, int64_t M, int64_t F,
                              cudaStream_t s);

// dg = dh u act'(g), du = dh act(g); all of one type.
cudaError_t gated_slopes_launch(const void *dh, int64_t lddh, const void *g, int64_t ldg,
                                const void *u, int64_t ldu, void *dg, int64_t lddg, void *du,
                                int64_t lddu, int dtype, int act, int64_t M, int64_t F,
                                cudaStream_t s);

// dz = dy act'(pre) (dy, pre: grad_dtype; dz: dz_dtype, or null) and dbias = its column sums
// (or null). `partials`: column_partials_bytes(M, N, 1) of workspace when dbias is given.
cudaError_t epilogue_slopes_launch(const void *dy, int64_t lddy, const void *pre, int64_t ld_pre,
                                   int grad_dtype, int act, void *dz, int64_t lddz, int dz_dtype,
                                   void *dbias, int bias_dtype, float *partials, int64_t M,
                                   int64_t N, int sm_count, cudaStream_t s);

// y = a + b in fp32, rounded to out_dtype (M x N; y's rows may be a's).
cudaError_t add_rows_launch(const float *a, int64_t lda, const float *b, int64_t ldb, void *y,
                            int64_t ldy, int out_dtype, int64_t M, int64_t N, cudaStream_t s);

// Column sums in two steps: each CTA adds up a band of rows into `partials`
// ([band][sums][N] fp32), a second kernel adds the bands in their order.
int64_t column_bands(int64_t M, int64_t N, int sm_count);
inline size_t column_partials_bytes(int64_t M, int64_t N, int sums, int sm_count) {
  return static_cast<size_t>(column_bands(M, N, sm_count) * N * sums) * sizeof(float);
}
// out[j] = sum over the bands of partials[(b * sums + which) * N + j], for `sums` outputs
// (out1 null: one).
cudaError_t column_finish_launch(const float *partials, int64_t bands, int sums, void *out0,
                                 void *out1, int dtype, int64_t N, cudaStream_t s);

cudaError_t layer_norm_launch(const void *x, int64_t ldx, int in_dtype, const void *weight,
                              const void *bias, int param_dtype, void *y, int64_t ldy,
                              int out_dtype, float *mean, float *rstd, float eps, int64_t M,
                              int64_t N, int sm_count, cudaStream_t s);

// Workspace of the backward pass (one_type: dy has x's type).
size_t layer_norm_backward_bytes(int64_t M, int64_t N, bool one_type, int sm_count);
cudaError_t layer_norm_backward_launch(const void *dy, int64_t lddy, int grad_dtype, const void *x,
                                       int64_t ldx, int in_dtype, const void *weight,
                                       int param_dtype, const float *mean, const float *rstd,
                                       void *dx, int64_t lddx, void *dweight, void *dbias,
                                       void *workspace, int64_t M, int64_t N, int sm_count,
                                       int *launches, cudaStream_t s);

}  // namespace ff
}  // namespace gemm_gb300
