// expert_internal.h -- launchers of the kernels behind the operators of experts and of dropout,
// shared by their C entries (experts.cu) and the kernels' translation units. Internal to the
// library.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace gemm_gb300 {
namespace ff {

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxSorted = int64_t{1} << 26;  // ids of a call (the work grows with their square)
// A token's choices: the row kernels step through them by warps, 32 at a time, in 32 bits.
constexpr int64_t kMaxChoices = INT32_MAX - 31;
// Rows and features of the products: the kernels round them up to whole tiles and boxes (256 at most,
// and 256 past a tile's start) in 32 bits.
constexpr int64_t kMaxProductSize = INT32_MAX - 511;

// Workspace of expert_sort_launch (0 when one CTA takes all ids).
size_t expert_sort_bytes(int64_t n, int64_t experts);
// position and offsets of `tokens` x `k` expert ids (8 or 4 bytes each), rows ld_ids apart.
cudaError_t expert_sort_launch(const void *ids, int64_t ld_ids, bool wide, int64_t tokens, int64_t k,
                               int64_t experts, int32_t *position, int32_t *offsets,
                               void *workspace, int *launches, cudaStream_t s);

// y[position[t, j]] = x[t] for the positions inside [0, rows).
cudaError_t expert_gather_launch(const void *x, int64_t ldx, const int32_t *position, void *y,
                                 int64_t ldy, int es, int64_t tokens, int64_t k, int64_t rows,
                                 int64_t N, cudaStream_t s);

// y[t] = sum_j w[t, j] z[position[t, j]] + residual[t] (w null: 1; residual null: 0).
cudaError_t expert_combine_launch(const void *z, int64_t ldz, int in_dtype, const int32_t *position,
                                  const void *w, int w_dtype, const void *residual, int64_t ldr,
                                  void *y, int64_t ldy, int out_dtype, int64_t tokens, int64_t k,
                                  int64_t rows, int64_t N, int sm_count, int *status, uint64_t timeout_ns,
                                  bool stall, cudaStream_t s);
// The same by bulk copies: rows that start on 16-byte boundaries and are a multiple of eight long, of
// sizes that fit. `stall`: no copy is issued, the waits (timeout_ns) end in the status.
bool expert_combine_bulk_fits(int64_t tokens, int64_t k, int64_t N, int in_dtype, int out_dtype,
                              bool residual, int sm_count);
cudaError_t expert_combine_bulk_launch(const void *z, int64_t ldz, int in_dtype, const int32_t *position,
                                       const void *w, int w_dtype, const void *residual, int64_t ldr,
                                       void *y, int64_t ldy, int out_dtype, int64_t tokens, int64_t k,
                                       int64_t rows, int64_t N, int sm_count, int *status,
                                       uint64_t timeout_ns, bool stall, cudaStream_t s);

// dz[position[t, j]] = w[t, j] dy[t] (or null), dw[t, j] = dy[t] . z[position[t, j]] (or null).
cudaError_t expert_combine_backward_launch(const void *dy, int64_t lddy, int grad_dtype,
                                           const void *z, int64_t ldz, const int32_t *position,
                                           const void *w, int w_dtype, void *dz, int64_t lddz,
                                           int in_dtype, void *dw, int64_t tokens, int64_t k,
                                           int64_t rows, int64_t N, int sm_count, cudaStream_t s);

// Zeros in the rows of all experts (an empty sum).
cudaError_t expert_zero_launch(void *y, int64_t ldy, int es, const int32_t *offsets, int64_t experts,
                               int64_t rows, int64_t N, cudaStream_t s);

// fp32: h = act(g) * u for the rows of all experts; h may be g.
cudaError_t expert_gated_rows_launch(const float *g, int64_t ldg, const float *u, int64_t ldu, float *h,
                                     int64_t ldh, int act, const int32_t *offsets, int64_t experts,
                                     int64_t rows, int64_t F, cudaStream_t s);

// Copies `count` matrices of `lines` lines of `len` 16-bit elements (lines ld apart, matrices stride
// apart, of any alignment) to lines to_ld apart that follow one another from a 16-byte boundary
// (to_ld: a multiple of 8, at least len); with offsets only those whose experts have rows.
cudaError_t expert_stage_launch(const void *src, int64_t ld, int64_t stride, int64_t lines, int64_t count,
                                int64_t len, void *dst, int64_t to_ld, const int32_t *offsets, cudaStream_t s);

// y = x * mask * scale + residual (null: 0); key: two 64-bit words on the device.
cudaError_t dropout_launch(const void *x, int64_t ldx, const void *residual, int64_t ldr, void *y,
                           int64_t ldy, int dtype, uint32_t threshold, float scale,
                           const uint64_t *key, int64_t M, int64_t N, cudaStream_t s);

}  // namespace ff
}  // namespace gemm_gb300
