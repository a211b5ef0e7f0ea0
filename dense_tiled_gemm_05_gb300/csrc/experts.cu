// experts.cu -- the C ABI of the operators of experts (the order of tokens by expert, rows into
// that order and back) and of dropout: argument checks and launches.
#include <cmath>

#include "api_internal.h"
#include "expert_internal.h"
#include "ff_checks.h"

using namespace gemm_gb300;
using namespace gemm_gb300::api;
using ff::bad_matrix;
using ff::disjoint;
using ff::launched;
using ff::matrix_span;
using ff::misaligned;
using ff::Span;
using ff::vector_span;

namespace {

bool too_large(int64_t tokens, int64_t k, int64_t rows, int64_t N) {
  return tokens > INT32_MAX || k > INT32_MAX || rows > INT32_MAX || N > INT32_MAX ||
         tokens * k > INT32_MAX;
}

}  // namespace

extern "C" {

GEMM_API gemm_status_t gemm_expert_sort(gemm_handle_t h, int64_t tokens, int64_t k,
                                        int64_t experts, const void *ids, int64_t ld_ids,
                                        int32_t id_bytes, int32_t *position, int32_t *offsets,
                                        void *cuda_stream) {
  if (!h || tokens < 0 || k < 0 || experts < 1 || (id_bytes != 4 && id_bytes != 8) || !offsets)
    return GEMM_ERR_INVALID_ARG;
  if (bad_matrix(ids, tokens, k, ld_ids, GEMM_ROW_MAJOR) || (tokens > 0 && k > 0 && !position))
    return GEMM_ERR_INVALID_ARG;
  if (experts > ff::kMaxExperts || too_large(tokens, k, 0, 0)) return GEMM_ERR_UNSUPPORTED;
  if (misaligned(ids, id_bytes) || misaligned(position, 4) || misaligned(offsets, 4))
    return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {vector_span(position, tokens * k, 4), vector_span(offsets, experts + 1, 4)};
  const Span ins[] = {matrix_span(ids, tokens, k, ld_ids, GEMM_ROW_MAJOR, id_bytes)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const gemm_status_t st = reserve(h, h->ff, ff::expert_sort_bytes(tokens * k, experts), s);
  if (st != GEMM_OK) return st;
  int launches = 0;
  const cudaError_t e = ff::expert_sort_launch(ids, ld_ids, id_bytes == 8, tokens, k, experts,
                                               position, offsets, h->ff.ptr, &launches, s);
  return launched(h, e, "expert sort launch", launches);
}

GEMM_API gemm_status_t gemm_expert_gather(gemm_handle_t h, int64_t tokens, int64_t k, int64_t N,
                                          const void *X, int64_t ldx, const int32_t *position,
                                          int64_t rows, void *Y, int64_t ldy, gemm_dtype_t dtype,
                                          void *cuda_stream) {
  if (!h || tokens < 0 || k < 0 || N < 0 || rows < 0 || !valid_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 || k == 0 || N == 0 || rows == 0) return GEMM_OK;
  if (bad_matrix(X, tokens, N, ldx, GEMM_ROW_MAJOR) || bad_matrix(Y, rows, N, ldy, GEMM_ROW_MAJOR) ||
      !position)
    return GEMM_ERR_INVALID_ARG;
  if (too_large(tokens, k, rows, N)) return GEMM_ERR_UNSUPPORTED;
  const int es = esize_of(dtype);
  if (misaligned(X, es) || misaligned(Y, es) || misaligned(position, 4)) return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(Y, rows, N, ldy, GEMM_ROW_MAJOR, es)};
  const Span ins[] = {matrix_span(X, tokens, N, ldx, GEMM_ROW_MAJOR, es),
                      vector_span(position, tokens * k, 4)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  return launched(h, ff::expert_gather_launch(X, ldx, position, Y, ldy, es, tokens, k, rows, N,
                                              static_cast<cudaStream_t>(cuda_stream)),
                  "expert gather launch");
}

GEMM_API gemm_status_t gemm_expert_combine(gemm_handle_t h, int64_t tokens, int64_t k, int64_t N,
                                           const void *Z, int64_t ldz, int64_t rows,
                                           const int32_t *position, const void *weights,
                                           gemm_dtype_t weight_dtype, const void *residual,
                                           int64_t ld_residual, void *Y, int64_t ldy,
                                           gemm_dtype_t in_dtype, gemm_dtype_t out_dtype,
                                           void *cuda_stream) {
  if (!h || tokens < 0 || k < 0 || N < 0 || rows < 0 || !valid_dtype(in_dtype) ||
      !valid_dtype(out_dtype) || (weights && !valid_dtype(weight_dtype)))
    return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 || N == 0) return GEMM_OK;
  if (bad_matrix(Y, tokens, N, ldy, GEMM_ROW_MAJOR) || (k > 0 && !position) ||
      (k > 0 && bad_matrix(Z, rows, N, ldz, GEMM_ROW_MAJOR)) || (residual && ld_residual < N))
    return GEMM_ERR_INVALID_ARG;
  if (too_large(tokens, k, rows, N)) return GEMM_ERR_UNSUPPORTED;
  const int is = esize_of(in_dtype), os = esize_of(out_dtype);
  const int ws = weights ? esize_of(weight_dtype) : 1;
  if (misaligned(Z, is) || misaligned(Y, os) || misaligned(residual, os) || misaligned(position, 4) ||
      misaligned(weights, ws))
    return GEMM_ERR_ALIGNMENT;
  const bool in_place = residual == Y && ld_residual == ldy;
  const Span outs[] = {matrix_span(Y, tokens, N, ldy, GEMM_ROW_MAJOR, os)};
  const Span ins[] = {matrix_span(Z, rows, N, ldz, GEMM_ROW_MAJOR, is),
                      in_place ? Span{} : matrix_span(residual, tokens, N, ld_residual, GEMM_ROW_MAJOR, os),
                      vector_span(position, tokens * k, 4), vector_span(weights, tokens * k, ws)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  return launched(h, ff::expert_combine_launch(Z, ldz, in_dtype, position, weights,
                                               weights ? weight_dtype : GEMM_F32, residual,
                                               ld_residual, Y, ldy, out_dtype, tokens, k, rows, N,
                                               static_cast<cudaStream_t>(cuda_stream)),
                  "expert combine launch");
}

GEMM_API gemm_status_t gemm_expert_combine_backward(
    gemm_handle_t h, int64_t tokens, int64_t k, int64_t N, const void *dY, int64_t lddy,
    const void *Z, int64_t ldz, int64_t rows, const int32_t *position, const void *weights,
    gemm_dtype_t weight_dtype, void *dZ, int64_t lddz, void *dweights, gemm_dtype_t in_dtype,
    gemm_dtype_t out_dtype, void *cuda_stream) {
  if (!h || tokens < 0 || k < 0 || N < 0 || rows < 0 || !valid_dtype(in_dtype) ||
      !valid_dtype(out_dtype) || ((weights || dweights) && !valid_dtype(weight_dtype)))
    return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 || k == 0 || (!dZ && !dweights)) return GEMM_OK;
  if (bad_matrix(dY, tokens, N, lddy, GEMM_ROW_MAJOR) || !position ||
      (dZ && bad_matrix(dZ, rows, N, lddz, GEMM_ROW_MAJOR)) ||
      (dweights && bad_matrix(Z, rows, N, ldz, GEMM_ROW_MAJOR)))
    return GEMM_ERR_INVALID_ARG;
  if (too_large(tokens, k, rows, N)) return GEMM_ERR_UNSUPPORTED;
  const int is = esize_of(in_dtype), os = esize_of(out_dtype);
  const int ws = weights || dweights ? esize_of(weight_dtype) : 1;
  if (misaligned(dY, os) || (dweights && misaligned(Z, is)) || misaligned(dZ, is) ||
      misaligned(position, 4) || misaligned(weights, ws) || misaligned(dweights, ws))
    return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(dZ, rows, N, lddz, GEMM_ROW_MAJOR, is),
                       vector_span(dweights, tokens * k, ws)};
  const Span ins[] = {matrix_span(dY, tokens, N, lddy, GEMM_ROW_MAJOR, os),
                      dweights ? matrix_span(Z, rows, N, ldz, GEMM_ROW_MAJOR, is) : Span{},
                      vector_span(position, tokens * k, 4), vector_span(weights, tokens * k, ws)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  return launched(h, ff::expert_combine_backward_launch(
                         dY, lddy, out_dtype, Z, ldz, position, weights,
                         weights || dweights ? weight_dtype : GEMM_F32, dZ, lddz, in_dtype, dweights,
                         tokens, k, rows, N, h->sm_count, static_cast<cudaStream_t>(cuda_stream)),
                  "expert combine backward launch");
}

GEMM_API gemm_status_t gemm_dropout(gemm_handle_t h, int64_t M, int64_t N, const void *X,
                                    int64_t ldx, const void *residual, int64_t ld_residual,
                                    void *Y, int64_t ldy, double p, const uint64_t *key,
                                    gemm_dtype_t dtype, void *cuda_stream) {
  if (!h || M < 0 || N < 0 || !valid_dtype(dtype) || !(p >= 0.0) || !(p < 1.0))
    return GEMM_ERR_INVALID_ARG;
  const uint32_t threshold = static_cast<uint32_t>(std::floor(65536.0 * p + 0.5));
  if (threshold > 65535u) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  if (bad_matrix(X, M, N, ldx, GEMM_ROW_MAJOR) || bad_matrix(Y, M, N, ldy, GEMM_ROW_MAJOR) ||
      (residual && ld_residual < N) || !key)
    return GEMM_ERR_INVALID_ARG;
  if (M > INT32_MAX || N > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
  const int es = esize_of(dtype);
  if (misaligned(X, es) || misaligned(residual, es) || misaligned(Y, es) || misaligned(key, 8))
    return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(Y, M, N, ldy, GEMM_ROW_MAJOR, es)};
  const Span ins[] = {X == Y && ldx == ldy ? Span{} : matrix_span(X, M, N, ldx, GEMM_ROW_MAJOR, es),
                      residual == Y && ld_residual == ldy
                          ? Span{}
                          : matrix_span(residual, M, N, ld_residual, GEMM_ROW_MAJOR, es),
                      vector_span(key, 2, 8)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const float scale = static_cast<float>(65536.0 / (65536.0 - threshold));
  return launched(h, ff::dropout_launch(X, ldx, residual, ld_residual, Y, ldy, dtype, threshold, scale,
                                        key, M, N, static_cast<cudaStream_t>(cuda_stream)),
                  "dropout launch");
}

}  // extern "C"
