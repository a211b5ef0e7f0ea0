// experts.cu -- the C ABI of the operators of experts (the order of tokens by expert, rows into
// that order and back, the experts' products) and of dropout: argument checks and launches.
#include <cmath>

#include "api_internal.h"
#include "expert_launch.h"
#include "ff_checks.h"

using namespace gemm_gb300;
using namespace gemm_gb300::api;
using ff::bad_matrix;
using ff::Carve;
using ff::disjoint;
using ff::launched;
using ff::matrix_span;
using ff::misaligned;
using ff::Span;
using ff::valid_act;
using ff::vector_span;

namespace {

bool too_large(int64_t tokens, int64_t k, int64_t rows, int64_t N) {
  return tokens > INT32_MAX || k > ff::kMaxChoices || rows > INT32_MAX || N > INT32_MAX ||
         tokens * k > INT32_MAX;
}

// Elements that the K x N weights of one expert span.
int64_t weight_span(int64_t K, int64_t N, int64_t ld, int layout) {
  return layout == GEMM_ROW_MAJOR ? (K - 1) * ld + N : (N - 1) * ld + K;
}
bool bad_weights(const void *W, int64_t experts, int64_t K, int64_t N, int64_t ld, int64_t stride,
                 int layout) {
  if (K == 0 || N == 0) return false;
  return bad_matrix(W, K, N, ld, layout) || (experts > 1 && stride < weight_span(K, N, ld, layout));
}
// All experts' weights. Two sets may be parts of one buffer: column ranges of the same lines (where
// experts are whole lines apart, so that all lines are multiples of ld from the first), or blocks of
// lines, expert by expert.
Span weights_span(const void *W, int64_t experts, int64_t K, int64_t N, int64_t ld, int64_t stride,
                  int layout, int es) {
  if (!W || K == 0 || N == 0) return Span{};
  Span s = matrix_span(W, K, N, ld, layout, es);  // the first expert's
  if (experts == 1) return s;
  s.block = s.hi - s.lo, s.block_pitch = static_cast<uintptr_t>(stride * es);
  s.hi += static_cast<uintptr_t>((experts - 1) * stride * es);
  if (stride % ld != 0) s.pitch = 0;
  return s;
}

// What the experts' products share: sizes and offsets.
gemm_status_t check_experts(gemm_handle_t h, int64_t experts, int64_t rows, int64_t N, int64_t K,
                            const int32_t *offsets, int dtype, int layout) {
  if (!h || experts < 1 || rows < 0 || N < 0 || K < 0 || !offsets || !valid_dtype(dtype) ||
      !valid_layout(layout))
    return GEMM_ERR_INVALID_ARG;
  if (experts > ff::kMaxExperts || rows > ff::kMaxProductSize || N > ff::kMaxProductSize ||
      K > ff::kMaxProductSize || 2 * N > INT32_MAX ||
      !ff::expert_tiles_fit(experts, rows, N > 0 ? N : 1, K > 0 ? K : 1))
    return GEMM_ERR_UNSUPPORTED;
  return misaligned(offsets, 4) ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

gemm_status_t zero_rows(gemm_handle_t h, void *Y, int64_t ld, int64_t rows, int64_t N, int es,
                        const int32_t *offsets, int64_t experts, cudaStream_t s) {
  if (!Y || rows == 0 || N == 0) return GEMM_OK;
  return launched(h, ff::expert_zero_launch(Y, ld, es, offsets, experts, rows, N, s), "expert zero launch");
}
// The experts' weight gradients without any row.
gemm_status_t zero_weights(gemm_handle_t h, void *D, int64_t experts, int64_t lines, int64_t len,
                           int64_t ld, int64_t stride, int dtype, cudaStream_t s) {
  const bool one = experts == 1 || stride == lines * ld;
  for (int64_t e = 0; e < (one ? 1 : experts); ++e) {
    const gemm_status_t st =
        launched(h, zero_fill_launch(static_cast<char *>(D) + e * stride * esize_of(dtype), ld,
                                     one ? experts * lines : lines, len, dtype, s), "zero fill");
    if (st != GEMM_OK) return st;
  }
  return GEMM_OK;
}

// dW of one product from its operands' rows.
gemm_status_t weight_gradient(gemm_handle_t h, const ff::ExpertOperand &X, const ff::ExpertOperand &dY,
                              int64_t experts, const int32_t *offsets, void *dW, int64_t ld,
                              int64_t stride, int dtype, int layout, cudaStream_t s) {
  const ff::ExpertOperand &A = layout == GEMM_ROW_MAJOR ? X : dY, &B = layout == GEMM_ROW_MAJOR ? dY : X;
  if (!dW || A.len == 0 || B.len == 0) return GEMM_OK;
  if (X.lines == 0) return zero_weights(h, dW, experts, A.len, B.len, ld, stride, dtype, s);
  ff::ExpertGrad q;
  q.experts = experts, q.rows = X.lines, q.offsets = offsets;
  q.A = A, q.B = B;
  q.dtype = dtype;
  q.D = dW, q.ldd = ld, q.stride_d = stride;
  return dtype == GEMM_F32 ? ff::run_expert_grad_f32(h, q, s) : ff::run_expert_grad(h, q, s);
}

int flip(int layout) { return layout == GEMM_ROW_MAJOR ? GEMM_COL_MAJOR : GEMM_ROW_MAJOR; }

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
  if (experts > ff::kMaxExperts || too_large(tokens, k, 0, 0) || tokens * k > ff::kMaxSorted)
    return GEMM_ERR_UNSUPPORTED;
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
                                               h->sm_count, h->status, h->timeout_us * 1000ull,
                                               (stall_flags(h->stall_producer) & kDebugStallProducer) != 0,
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

GEMM_API gemm_status_t gemm_run_expert(gemm_handle_t h, int64_t experts, int64_t rows, int64_t N,
                                       int64_t K, const void *X, int64_t ldx, const void *W,
                                       int64_t ldw, int64_t stride_w, const int32_t *offsets,
                                       void *Y, int64_t ldy, gemm_dtype_t dtype,
                                       gemm_layout_t w_layout, void *cuda_stream) {
  gemm_status_t st = check_experts(h, experts, rows, N, K, offsets, dtype, w_layout);
  if (st != GEMM_OK) return st;
  if (rows == 0 || N == 0) return GEMM_OK;
  if (bad_matrix(X, rows, K, ldx, GEMM_ROW_MAJOR) || bad_matrix(Y, rows, N, ldy, GEMM_ROW_MAJOR) ||
      bad_weights(W, experts, K, N, ldw, stride_w, w_layout))
    return GEMM_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (misaligned(X, es) || misaligned(W, es) || misaligned(Y, es)) return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(Y, rows, N, ldy, GEMM_ROW_MAJOR, es)};
  const Span ins[] = {matrix_span(X, rows, K, ldx, GEMM_ROW_MAJOR, es),
                      weights_span(W, experts, K, N, ldw, stride_w, w_layout, es),
                      vector_span(offsets, experts + 1, 4)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (K == 0) return zero_rows(h, Y, ldy, rows, N, es, offsets, experts, s);
  ff::ExpertProduct q;
  q.experts = experts, q.rows = rows, q.N = N, q.K = K, q.offsets = offsets;
  q.X = ff::expert_rows(X, ldx, rows, K);
  q.W = ff::expert_weights(W, ldw, stride_w, experts, K, N, w_layout);
  q.w_mn = w_layout == GEMM_ROW_MAJOR;
  q.dtype = dtype;
  q.C = Y, q.ldc = ldy;
  if (dtype == GEMM_F32) return ff::run_expert_f32(h, q, false, s);
  Carve carve;
  q.X.plan(&carve), q.W.plan(&carve);
  st = reserve(h, h->ff, carve.bytes, s);
  char *buf = static_cast<char *>(h->ff.ptr);
  if (st == GEMM_OK) st = q.X.stage(h, buf, s);
  if (st == GEMM_OK) st = q.W.stage(h, buf, s, offsets);
  return st == GEMM_OK ? ff::run_expert(h, q, s) : st;
}

GEMM_API gemm_status_t gemm_run_expert_backward(
    gemm_handle_t h, int64_t experts, int64_t rows, int64_t N, int64_t K, const void *dY,
    int64_t lddy, const void *X, int64_t ldx, const void *W, int64_t ldw, int64_t stride_w,
    const int32_t *offsets, void *dX, int64_t lddx, void *dW, int64_t lddw, int64_t stride_dw,
    gemm_dtype_t dtype, gemm_layout_t w_layout, void *cuda_stream) {
  gemm_status_t st = check_experts(h, experts, rows, N, K, offsets, dtype, w_layout);
  if (st != GEMM_OK) return st;
  if (bad_matrix(dY, rows, N, lddy, GEMM_ROW_MAJOR) ||
      (dX && (bad_matrix(dX, rows, K, lddx, GEMM_ROW_MAJOR) ||
              bad_weights(W, experts, K, N, ldw, stride_w, w_layout))) ||
      (dW && (bad_matrix(X, rows, K, ldx, GEMM_ROW_MAJOR) ||
              bad_weights(dW, experts, K, N, lddw, stride_dw, w_layout))))
    return GEMM_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (misaligned(dY, es) || (dW && misaligned(X, es)) || (dX && misaligned(W, es)) ||
      misaligned(dX, es) || misaligned(dW, es))
    return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(dX, rows, K, lddx, GEMM_ROW_MAJOR, es),
                       weights_span(dW, experts, K, N, lddw, stride_dw, w_layout, es)};
  const Span ins[] = {matrix_span(dY, rows, N, lddy, GEMM_ROW_MAJOR, es),
                      dW ? matrix_span(X, rows, K, ldx, GEMM_ROW_MAJOR, es) : Span{},
                      dX ? weights_span(W, experts, K, N, ldw, stride_w, w_layout, es) : Span{},
                      vector_span(offsets, experts + 1, 4)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  if (!dX && !dW) return GEMM_OK;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool make_dx = dX && rows > 0 && K > 0 && N > 0;
  ff::ExpertOperand xs = ff::expert_rows(X, ldx, rows, K), ys = ff::expert_rows(dY, lddy, rows, N);
  ff::ExpertOperand ws = ff::expert_weights(W, ldw, stride_w, experts, K, N, w_layout);
  const bool f32 = dtype == GEMM_F32;
  Carve carve;
  if (!f32) ys.plan(&carve);
  if (!f32 && dW) xs.plan(&carve);
  if (!f32 && make_dx) ws.plan(&carve);
  st = reserve(h, h->ff, carve.bytes, s);
  char *buf = static_cast<char *>(h->ff.ptr);
  if (st == GEMM_OK) st = ys.stage(h, buf, s);
  if (st == GEMM_OK) st = xs.stage(h, buf, s);
  if (st == GEMM_OK) st = ws.stage(h, buf, s, offsets);
  if (st != GEMM_OK) return st;
  if (make_dx) {
    ff::ExpertProduct q;
    q.experts = experts, q.rows = rows, q.N = K, q.K = N, q.offsets = offsets;
    q.X = ys, q.W = ws;
    q.w_mn = flip(w_layout) == GEMM_ROW_MAJOR;
    q.dtype = dtype;
    q.C = dX, q.ldc = lddx;
    st = f32 ? ff::run_expert_f32(h, q, false, s) : ff::run_expert(h, q, s);
  } else if (dX) {
    st = zero_rows(h, dX, lddx, rows, K, es, offsets, experts, s);
  }
  if (st != GEMM_OK) return st;
  return weight_gradient(h, xs, ys, experts, offsets, dW, lddw, stride_dw, dtype, w_layout, s);
}

GEMM_API gemm_status_t gemm_run_expert_gated(
    gemm_handle_t h, int64_t experts, int64_t rows, int64_t F, int64_t K, const void *X,
    int64_t ldx, const void *Wg, int64_t ldwg, int64_t stride_wg, const void *Wu, int64_t ldwu,
    int64_t stride_wu, const int32_t *offsets, void *H, int64_t ldh, void *gate, int64_t ld_gate,
    void *up, int64_t ld_up, gemm_dtype_t dtype, gemm_layout_t w_layout,
    gemm_activation_t activation, void *cuda_stream) {
  gemm_status_t st = check_experts(h, experts, rows, F, K, offsets, dtype, w_layout);
  if (st != GEMM_OK) return st;
  if (!valid_act(activation) || (gate == nullptr) != (up == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || F == 0) return GEMM_OK;
  if (bad_matrix(X, rows, K, ldx, GEMM_ROW_MAJOR) || bad_matrix(H, rows, F, ldh, GEMM_ROW_MAJOR) ||
      bad_weights(Wg, experts, K, F, ldwg, stride_wg, w_layout) ||
      bad_weights(Wu, experts, K, F, ldwu, stride_wu, w_layout) || (gate && (ld_gate < F || ld_up < F)))
    return GEMM_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  for (const void *p : {X, Wg, Wu, static_cast<const void *>(H), static_cast<const void *>(gate),
                        static_cast<const void *>(up)})
    if (misaligned(p, es)) return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(H, rows, F, ldh, GEMM_ROW_MAJOR, es),
                       matrix_span(gate, rows, F, ld_gate, GEMM_ROW_MAJOR, es),
                       matrix_span(up, rows, F, ld_up, GEMM_ROW_MAJOR, es)};
  const Span ins[] = {matrix_span(X, rows, K, ldx, GEMM_ROW_MAJOR, es),
                      weights_span(Wg, experts, K, F, ldwg, stride_wg, w_layout, es),
                      weights_span(Wu, experts, K, F, ldwu, stride_wu, w_layout, es),
                      vector_span(offsets, experts + 1, 4)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (K == 0) {  // g = u = 0, and so h
    st = zero_rows(h, H, ldh, rows, F, es, offsets, experts, s);
    if (st == GEMM_OK) st = zero_rows(h, gate, ld_gate, rows, F, es, offsets, experts, s);
    return st == GEMM_OK ? zero_rows(h, up, ld_up, rows, F, es, offsets, experts, s) : st;
  }
  ff::ExpertProduct q;
  q.gated = true;
  q.experts = experts, q.rows = rows, q.N = F, q.K = K, q.offsets = offsets;
  q.X = ff::expert_rows(X, ldx, rows, K);
  q.W = ff::expert_weights(Wg, ldwg, stride_wg, experts, K, F, w_layout);
  q.W2 = ff::expert_weights(Wu, ldwu, stride_wu, experts, K, F, w_layout);
  q.w_mn = w_layout == GEMM_ROW_MAJOR;
  q.dtype = dtype, q.act = activation;
  q.C = H, q.ldc = ldh;
  q.pre = gate, q.ld_pre = ld_gate, q.pre2 = up, q.ld_pre2 = ld_up;
  if (dtype == GEMM_F32) {
    // g goes to gate or, where that is not asked for, to H, and h = act(g) u takes its place; u goes to
    // up or to the handle's buffer.
    const int64_t ld_u = up ? ld_up : F, ld_g = gate ? ld_gate : ldh;
    if (!up) st = reserve(h, h->ff, static_cast<size_t>(rows * F) * sizeof(float), s);
    if (st != GEMM_OK) return st;
    void *g32 = gate ? gate : H, *u32 = up ? up : h->ff.ptr;
    q.C = g32, q.ldc = ld_g;
    st = ff::run_expert_f32(h, q, false, s);
    q.W = q.W2, q.C = u32, q.ldc = ld_u;
    if (st == GEMM_OK) st = ff::run_expert_f32(h, q, false, s);
    if (st != GEMM_OK) return st;
    return launched(h, ff::expert_gated_rows_launch(static_cast<const float *>(g32), ld_g,
                                                    static_cast<const float *>(u32), ld_u,
                                                    static_cast<float *>(H), ldh, activation, offsets,
                                                    experts, rows, F, s),
                    "expert gated rows launch");
  }
  Carve carve;
  q.X.plan(&carve), q.W.plan(&carve), q.W2.plan(&carve);
  st = reserve(h, h->ff, carve.bytes, s);
  char *buf = static_cast<char *>(h->ff.ptr);
  if (st == GEMM_OK) st = q.X.stage(h, buf, s);
  if (st == GEMM_OK) st = q.W.stage(h, buf, s, offsets);
  if (st == GEMM_OK) st = q.W2.stage(h, buf, s, offsets);
  return st == GEMM_OK ? ff::run_expert(h, q, s) : st;
}

GEMM_API gemm_status_t gemm_run_expert_gated_backward(
    gemm_handle_t h, int64_t experts, int64_t rows, int64_t F, int64_t K, const void *dH,
    int64_t lddh, const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, const void *X,
    int64_t ldx, const void *Wg, int64_t ldwg, int64_t stride_wg, const void *Wu, int64_t ldwu,
    int64_t stride_wu, const int32_t *offsets, void *dX, int64_t lddx, void *dWg, int64_t lddwg,
    int64_t stride_dwg, void *dWu, int64_t lddwu, int64_t stride_dwu, gemm_dtype_t dtype,
    gemm_layout_t w_layout, gemm_activation_t activation, void *cuda_stream) {
  gemm_status_t st = check_experts(h, experts, rows, F, K, offsets, dtype, w_layout);
  if (st != GEMM_OK) return st;
  if (!valid_act(activation)) return GEMM_ERR_INVALID_ARG;
  const bool weights = dWg || dWu;
  if (bad_matrix(dH, rows, F, lddh, GEMM_ROW_MAJOR) || bad_matrix(gate, rows, F, ld_gate, GEMM_ROW_MAJOR) ||
      bad_matrix(up, rows, F, ld_up, GEMM_ROW_MAJOR) ||
      (weights && bad_matrix(X, rows, K, ldx, GEMM_ROW_MAJOR)) ||
      (dWg && bad_weights(dWg, experts, K, F, lddwg, stride_dwg, w_layout)) ||
      (dWu && bad_weights(dWu, experts, K, F, lddwu, stride_dwu, w_layout)) ||
      (dX && (bad_matrix(dX, rows, K, lddx, GEMM_ROW_MAJOR) ||
              bad_weights(Wg, experts, K, F, ldwg, stride_wg, w_layout) ||
              bad_weights(Wu, experts, K, F, ldwu, stride_wu, w_layout))))
    return GEMM_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  for (const void *p : {dH, gate, up, weights ? X : nullptr, dX ? Wg : nullptr, dX ? Wu : nullptr,
                        static_cast<const void *>(dX), static_cast<const void *>(dWg),
                        static_cast<const void *>(dWu)})
    if (misaligned(p, es)) return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(dX, rows, K, lddx, GEMM_ROW_MAJOR, es),
                       weights_span(dWg, experts, K, F, lddwg, stride_dwg, w_layout, es),
                       weights_span(dWu, experts, K, F, lddwu, stride_dwu, w_layout, es)};
  const Span ins[] = {matrix_span(dH, rows, F, lddh, GEMM_ROW_MAJOR, es),
                      matrix_span(gate, rows, F, ld_gate, GEMM_ROW_MAJOR, es),
                      matrix_span(up, rows, F, ld_up, GEMM_ROW_MAJOR, es),
                      weights ? matrix_span(X, rows, K, ldx, GEMM_ROW_MAJOR, es) : Span{},
                      dX ? weights_span(Wg, experts, K, F, ldwg, stride_wg, w_layout, es) : Span{},
                      dX ? weights_span(Wu, experts, K, F, ldwu, stride_wu, w_layout, es) : Span{},
                      vector_span(offsets, experts + 1, 4)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  if (!dX && !weights) return GEMM_OK;
  DeviceGuard guard(h->device);
  if (!guard.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool make_dx = dX && rows > 0 && K > 0 && F > 0;
  // dg | du side by side, on 16-byte boundaries
  const int64_t Fp = round_up(F, 8), ldd = 2 * Fp;
  ff::ExpertOperand xs = ff::expert_rows(X, ldx, rows, K);
  ff::ExpertOperand wg = ff::expert_weights(Wg, ldwg, stride_wg, experts, K, F, w_layout);
  ff::ExpertOperand wu = ff::expert_weights(Wu, ldwu, stride_wu, experts, K, F, w_layout);
  const bool f32 = dtype == GEMM_F32;
  Carve carve;
  const size_t d_off = carve.take(rows * ldd, es);
  if (!f32 && weights) xs.plan(&carve);
  if (!f32 && make_dx) wg.plan(&carve), wu.plan(&carve);
  st = reserve(h, h->ff, carve.bytes, s);
  if (st != GEMM_OK) return st;
  char *buf = static_cast<char *>(h->ff.ptr);
  char *dg = buf + d_off, *du = dg + Fp * es;
  if (rows > 0 && F > 0) {
    st = launched(h, ff::gated_slopes_launch(dH, lddh, gate, ld_gate, up, ld_up, dg, ldd, du, ldd,
                                             dtype, activation, rows, F, s),
                  "gated backward launch");
    if (st != GEMM_OK) return st;
  }
  st = xs.stage(h, buf, s);
  if (st == GEMM_OK) st = wg.stage(h, buf, s, offsets);
  if (st == GEMM_OK) st = wu.stage(h, buf, s, offsets);
  if (st != GEMM_OK) return st;
  const ff::ExpertOperand gs = ff::expert_rows(dg, ldd, rows, F), us = ff::expert_rows(du, ldd, rows, F);
  if (make_dx) {
    ff::ExpertProduct q;
    q.second = true;
    q.experts = experts, q.rows = rows, q.N = K, q.K = F, q.offsets = offsets;
    q.X = gs, q.W = wg, q.X2 = us, q.W2 = wu;
    q.w_mn = flip(w_layout) == GEMM_ROW_MAJOR;
    q.dtype = dtype;
    q.C = dX, q.ldc = lddx;
    if (f32) {
      st = ff::run_expert_f32(h, q, false, s);
      q.X = us, q.W = wu;
      if (st == GEMM_OK) st = ff::run_expert_f32(h, q, true, s);
    } else {
      st = ff::run_expert(h, q, s);
    }
  } else if (dX) {
    st = zero_rows(h, dX, lddx, rows, K, es, offsets, experts, s);
  }
  if (st == GEMM_OK)
    st = weight_gradient(h, xs, gs, experts, offsets, dWg, lddwg, stride_dwg, dtype, w_layout, s);
  if (st == GEMM_OK)
    st = weight_gradient(h, xs, us, experts, offsets, dWu, lddwu, stride_dwu, dtype, w_layout, s);
  return st;
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
