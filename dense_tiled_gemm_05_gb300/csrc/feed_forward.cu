// feed_forward.cu -- the C ABI of the feed-forward operators: products with an epilogue, the
// gated pair of projections, layer norm, and their backward passes. Argument checks, the
// choice of kernels, and the handle's buffer they share; the products that stand alone in
// the backward passes go through the planner like any gemm_run_ex call.
#include <cmath>

#include "api_internal.h"
#include "ff_launch.h"

using namespace gemm_gb300;
using namespace gemm_gb300::api;
using ff::Carve;

namespace {

bool valid_act(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SIGMOID; }

// A buffer of a call: the bytes it spans and, for a matrix, its line pitch and the bytes of a
// line, to keep outputs off inputs and each other.
struct Span {
  uintptr_t lo = 0, hi = 0;  // empty: lo == hi
  uintptr_t pitch = 0, line = 0;
  bool meets(const Span &o) const {
    if (!(lo < o.hi && o.lo < hi)) return false;
    // column ranges of one wider matrix share a span, but no element
    if (pitch == 0 || pitch != o.pitch) return true;
    const uintptr_t d = (lo < o.lo ? o.lo - lo : pitch - (lo - o.lo) % pitch) % pitch;
    return d < line || d + o.line > pitch;
  }
};

Span matrix_span(const void *p, int64_t rows, int64_t cols, int64_t ld, int layout, int es) {
  Span s;
  if (!p || rows <= 0 || cols <= 0) return s;
  span_of(p, rows, cols, ld, layout, es, &s.lo, &s.hi);
  s.pitch = static_cast<uintptr_t>(ld * es);
  s.line = static_cast<uintptr_t>((layout == GEMM_ROW_MAJOR ? cols : rows) * es);
  return s;
}
Span vector_span(const void *p, int64_t n, int es) {
  return matrix_span(p, 1, n, n, GEMM_ROW_MAJOR, es);
}

// Outputs may meet neither inputs nor each other.
template <int NO, int NI>
bool disjoint(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (outs[i].meets(outs[j])) return false;
    for (int j = 0; j < NI; ++j)
      if (outs[i].meets(ins[j])) return false;
  }
  return true;
}

bool misaligned(const void *p, int es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

// A row-major or column-major operand of a call that is used: pointer and leading dimension.
bool bad_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int layout) {
  if (rows == 0 || cols == 0) return false;
  return !p || ld < (layout == GEMM_ROW_MAJOR ? cols : rows);
}

// One product (its argument checks are the caller's own): few tokens and small exact fp32
// products on the fused operators' kernels, others through the planner, whose kernels for many
// tokens have no epilogue to make room for (1 x 4096 x 4096 bf16 on one GB300: 9.1 us against
// the planner's 21.6, 64 tokens 12.4 against 21.6). Not where the caller steers the planner by
// options or gemm_tune, and not where the fused kernels would have to stage an operand: the
// handle's buffer may hold this one's.
gemm_status_t product(gemm_handle_t h, const Problem &P, cudaStream_t s) {
  const bool f32 = P.in_dtype == GEMM_F32;
  if (P.precision != (f32 ? GEMM_PREC_TF32 : GEMM_PREC_F16_ACC) && !options_steer(h, P)) {
    ff::FusedProduct q;
    q.M = P.M, q.N = P.N, q.K = P.K;
    q.X.ptr = P.A, q.X.ld = P.lda, q.X.layout = P.a_layout;
    q.W.ptr = P.B, q.W.ld = P.ldb, q.W.layout = P.b_layout;
    q.in_dtype = P.in_dtype, q.out_dtype = P.out_dtype;
    q.C = P.C, q.ldc = P.ldc;
    Carve none;
    if (ff::plan_fused(h, &q, &none) && none.bytes == 0 && q.kind != ff::FusedProduct::kPair)
      return ff::run_fused(h, q, nullptr, s);
  }
  Plan pl;
  const gemm_status_t st = make_plan(P, options_for(h, P), h->sm_count, &pl);
  return st == GEMM_OK ? execute(h, P, pl, s) : st;
}

gemm_status_t launched(gemm_handle_t h, cudaError_t e, const char *what, int n = 1) {
  if (e != cudaSuccess) return cuda_fail(e, what);
  h->launches += static_cast<uint64_t>(n);
  return GEMM_OK;
}

int flip(int layout) { return layout == GEMM_ROW_MAJOR ? GEMM_COL_MAJOR : GEMM_ROW_MAJOR; }

// The operands' gradients of C = A @ B from dC (M x N, row-major, of in_dtype), each in its
// operand's layout. A gradient stored column-major is the transposed product, row-major.
gemm_status_t operand_gradients(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *dC,
                                int64_t lddc, const void *A, int64_t lda, int a_layout,
                                const void *B, int64_t ldb, int b_layout, void *dA, int64_t ldda,
                                void *dB, int64_t lddb, int dtype, int precision, cudaStream_t s) {
  gemm_status_t st = GEMM_OK;
  if (dA && M > 0 && K > 0) {
    const Problem P = a_layout == GEMM_ROW_MAJOR
                          ? Problem{M, K, N, dC, lddc, B, ldb, dA, ldda, dtype, dtype, precision,
                                    GEMM_ROW_MAJOR, flip(b_layout)}
                          : Problem{K, M, N, B, ldb, dC, lddc, dA, ldda, dtype, dtype, precision,
                                    b_layout, GEMM_COL_MAJOR};
    st = product(h, P, s);
    if (st != GEMM_OK) return st;
  }
  if (dB && N > 0 && K > 0) {
    const Problem P = b_layout == GEMM_ROW_MAJOR
                          ? Problem{K, N, M, A, lda, dC, lddc, dB, lddb, dtype, dtype, precision,
                                    flip(a_layout), GEMM_ROW_MAJOR}
                          : Problem{N, K, M, dC, lddc, A, lda, dB, lddb, dtype, dtype, precision,
                                    GEMM_COL_MAJOR, a_layout};
    st = product(h, P, s);
  }
  return st;
}

// Runs a product on the fused kernels when they take it.
gemm_status_t fused(gemm_handle_t h, ff::FusedProduct &q, bool *taken, cudaStream_t s) {
  Carve carve;
  *taken = ff::plan_fused(h, &q, &carve);
  if (!*taken) return GEMM_OK;
  const gemm_status_t st = reserve(h, h->ff, carve.bytes, s);
  return st == GEMM_OK ? ff::run_fused(h, q, static_cast<char *>(h->ff.ptr), s) : st;
}

gemm_status_t check_epilogue(const Problem &P, const gemm_epilogue_t &E) {
  if (!valid_act(E.activation)) return GEMM_ERR_INVALID_ARG;
  if (E.bias && !valid_dtype(E.bias_dtype)) return GEMM_ERR_INVALID_ARG;
  if (P.M == 0 || P.N == 0) return GEMM_OK;
  if ((E.residual && E.ld_residual < P.N) || (E.pre && E.ld_pre < P.N)) return GEMM_ERR_INVALID_ARG;
  const int os = esize_of(P.out_dtype), es = esize_of(P.in_dtype);
  if ((E.bias && misaligned(E.bias, esize_of(E.bias_dtype))) || misaligned(E.residual, os) ||
      misaligned(E.pre, os))
    return GEMM_ERR_ALIGNMENT;
  const Span c = matrix_span(P.C, P.M, P.N, P.ldc, GEMM_ROW_MAJOR, os);
  const Span r = matrix_span(E.residual, P.M, P.N, E.ld_residual, GEMM_ROW_MAJOR, os);
  const Span z = matrix_span(E.pre, P.M, P.N, E.ld_pre, GEMM_ROW_MAJOR, os);
  const Span a = P.K > 0 ? matrix_span(P.A, P.M, P.K, P.lda, P.a_layout, es) : Span{};
  const Span b = P.K > 0 ? matrix_span(P.B, P.K, P.N, P.ldb, P.b_layout, es) : Span{};
  const Span v = E.bias ? vector_span(E.bias, P.N, esize_of(E.bias_dtype)) : Span{};
  const bool in_place = E.residual == P.C && E.ld_residual == P.ldc;
  if ((!in_place && c.meets(r)) || c.meets(v) || c.meets(z) || z.meets(r) || z.meets(a) ||
      z.meets(b) || z.meets(v))
    return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

}  // namespace

extern "C" {

GEMM_API gemm_status_t gemm_run_epilogue(gemm_handle_t h, int64_t M, int64_t N, int64_t K,
                                         const void *A, int64_t lda, const void *B, int64_t ldb,
                                         void *C, int64_t ldc, gemm_dtype_t in_dtype,
                                         gemm_dtype_t out_dtype, gemm_precision_t precision_mode,
                                         gemm_layout_t a_layout, gemm_layout_t b_layout,
                                         const gemm_epilogue_t *epilogue, void *cuda_stream) {
  if (!h) return GEMM_ERR_INVALID_ARG;
  const Problem P{M, N, K, A, lda, B, ldb, C, ldc, in_dtype, out_dtype, precision_mode, a_layout,
                  b_layout};
  gemm_status_t st = check_args(P);
  if (st != GEMM_OK) return st;
  ff::Epilogue ep;
  if (epilogue) {
    st = check_epilogue(P, *epilogue);
    if (st != GEMM_OK) return st;
    ep.bias = epilogue->bias;
    ep.bias_dtype = epilogue->bias_dtype;
    ep.act = epilogue->activation;
    ep.residual = epilogue->residual;
    ep.ld_residual = epilogue->ld_residual;
    ep.pre = epilogue->pre;
    ep.ld_pre = epilogue->ld_pre;
  }
  if (M == 0 || N == 0) return GEMM_OK;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (ep.empty()) return product(h, P, s);
  if (precision_mode != GEMM_PREC_F16_ACC) {
    ff::FusedProduct q;
    q.M = M, q.N = N, q.K = K;
    q.X.ptr = A, q.X.ld = lda, q.X.layout = a_layout;
    q.W.ptr = B, q.W.ld = ldb, q.W.layout = b_layout;
    q.in_dtype = in_dtype, q.out_dtype = out_dtype;
    q.exact = precision_mode != GEMM_PREC_TF32;
    q.C = C, q.ldc = ldc;
    q.ep = ep;
    bool taken = false;
    st = fused(h, q, &taken, s);
    if (taken) return st;
  }
  // The product in fp32 first: into C itself when C is fp32 and not the residual, else into
  // the handle's buffer.
  Problem Q = P;
  Q.out_dtype = GEMM_F32;
  if (out_dtype != GEMM_F32 || ep.residual == C) {
    Q.ldc = round_up(N, 4);
    st = reserve(h, h->ff, static_cast<size_t>(M * Q.ldc) * sizeof(float), s);
    if (st != GEMM_OK) return st;
    Q.C = h->ff.ptr;
  }
  st = product(h, Q, s);
  if (st != GEMM_OK) return st;
  return launched(h, ff::epilogue_rows_launch(static_cast<const float *>(Q.C), Q.ldc, C, ldc,
                                              out_dtype, ep, M, N, s),
                  "epilogue launch");
}

GEMM_API gemm_status_t gemm_run_epilogue_backward(
    gemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *dY, int64_t lddy,
    const void *pre, int64_t ld_pre, const void *A, int64_t lda, const void *B, int64_t ldb,
    void *dA, int64_t ldda, void *dB, int64_t lddb, void *dbias, gemm_dtype_t bias_dtype,
    gemm_dtype_t in_dtype, gemm_dtype_t out_dtype, gemm_precision_t precision_mode,
    gemm_layout_t a_layout, gemm_layout_t b_layout, gemm_activation_t activation,
    void *cuda_stream) {
  if (!h || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || !valid_act(activation) ||
      !valid_layout(a_layout) || !valid_layout(b_layout) ||
      (dbias && !valid_dtype(bias_dtype)) || precision_mode < GEMM_PREC_DEFAULT ||
      precision_mode > GEMM_PREC_F16_ACC)
    return GEMM_ERR_INVALID_ARG;
  if (bad_matrix(dY, M, N, lddy, GEMM_ROW_MAJOR) ||
      (activation != GEMM_ACT_NONE && bad_matrix(pre, M, N, ld_pre, GEMM_ROW_MAJOR)) ||
      (dB && (bad_matrix(A, M, K, lda, a_layout) || bad_matrix(dB, K, N, lddb, b_layout))) ||
      (dA && (bad_matrix(B, K, N, ldb, b_layout) || bad_matrix(dA, M, K, ldda, a_layout))))
    return GEMM_ERR_INVALID_ARG;
  if (precision_mode == GEMM_PREC_F16_ACC ||
      (in_dtype != GEMM_F32 && precision_mode != GEMM_PREC_DEFAULT))
    return GEMM_ERR_UNSUPPORTED;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
  if (activation == GEMM_ACT_NONE) pre = nullptr;
  const int is = esize_of(in_dtype), os = esize_of(out_dtype);
  const int bs = dbias ? esize_of(bias_dtype) : 1;
  if (misaligned(dY, os) || misaligned(pre, os) || (dB && misaligned(A, is)) ||
      (dA && misaligned(B, is)) || misaligned(dA, is) || misaligned(dB, is) || misaligned(dbias, bs))
    return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(dA, M, K, ldda, a_layout, is),
                       matrix_span(dB, K, N, lddb, b_layout, is), vector_span(dbias, N, bs)};
  const Span ins[] = {matrix_span(dY, M, N, lddy, GEMM_ROW_MAJOR, os),
                      matrix_span(pre, M, N, ld_pre, GEMM_ROW_MAJOR, os),
                      dB ? matrix_span(A, M, K, lda, a_layout, is) : Span{},
                      dA ? matrix_span(B, K, N, ldb, b_layout, is) : Span{}};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  // dY is dz itself when there is no activation and it has the operands' type.
  const bool products = dA || dB;
  const bool make_dz = products && M > 0 && N > 0 && (pre || out_dtype != in_dtype);
  Carve carve;
  const int64_t lddz = round_up(N, 16 / is);
  const size_t dz_off = make_dz ? carve.take(M * lddz, is) : 0;
  const size_t part_off =
      dbias ? carve.take(static_cast<int64_t>(ff::column_partials_bytes(M, N, 1, h->sm_count)), 1) : 0;
  gemm_status_t st = reserve(h, h->ff, carve.bytes, s);
  if (st != GEMM_OK) return st;
  char *buf = static_cast<char *>(h->ff.ptr);
  void *dz = make_dz ? buf + dz_off : nullptr;
  if ((make_dz || dbias) && N > 0) {
    st = launched(h,
                  ff::epilogue_slopes_launch(dY, lddy, pre, ld_pre, out_dtype, activation, dz, lddz,
                                             in_dtype, dbias, dbias ? bias_dtype : GEMM_F32,
                                             reinterpret_cast<float *>(buf + part_off), M, N,
                                             h->sm_count, s),
                  "epilogue backward launch", dbias ? 2 : 1);
    if (st != GEMM_OK) return st;
  }
  return operand_gradients(h, M, N, K, make_dz ? dz : dY, make_dz ? lddz : lddy, A, lda, a_layout,
                           B, ldb, b_layout, dA, ldda, dB, lddb, in_dtype, precision_mode, s);
}

GEMM_API gemm_status_t gemm_run_gated(gemm_handle_t h, int64_t M, int64_t F, int64_t K,
                                      const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                                      const void *Wu, int64_t ldwu, void *H, int64_t ldh,
                                      void *gate, int64_t ld_gate, void *up, int64_t ld_up,
                                      gemm_dtype_t dtype, gemm_precision_t precision_mode,
                                      gemm_layout_t w_layout, gemm_activation_t activation,
                                      void *cuda_stream) {
  if (!h) return GEMM_ERR_INVALID_ARG;
  const Problem G{M, F, K, X, ldx, Wg, ldwg, H, ldh, dtype, dtype, precision_mode, GEMM_ROW_MAJOR,
                  w_layout};
  Problem U = G;
  U.B = Wu, U.ldb = ldwu;
  gemm_status_t st = check_args(G);
  if (st == GEMM_OK) st = check_args(U);
  if (st != GEMM_OK) return st;
  if (!valid_act(activation) || (gate == nullptr) != (up == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (precision_mode == GEMM_PREC_F16_ACC) return GEMM_ERR_UNSUPPORTED;
  if (M == 0 || F == 0) return GEMM_OK;
  const int es = esize_of(dtype);
  if (gate) {
    if (ld_gate < F || ld_up < F) return GEMM_ERR_INVALID_ARG;
    if (misaligned(gate, es) || misaligned(up, es)) return GEMM_ERR_ALIGNMENT;
    const Span outs[] = {matrix_span(H, M, F, ldh, GEMM_ROW_MAJOR, es),
                         matrix_span(gate, M, F, ld_gate, GEMM_ROW_MAJOR, es),
                         matrix_span(up, M, F, ld_up, GEMM_ROW_MAJOR, es)};
    const Span ins[] = {K > 0 ? matrix_span(X, M, K, ldx, GEMM_ROW_MAJOR, es) : Span{},
                        K > 0 ? matrix_span(Wg, K, F, ldwg, w_layout, es) : Span{},
                        K > 0 ? matrix_span(Wu, K, F, ldwu, w_layout, es) : Span{}};
    if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  }
  DeviceGuard guard(h->device);
  if (!guard.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  ff::FusedProduct q;
  q.gated = true;
  q.M = M, q.N = F, q.K = K;
  q.X.ptr = X, q.X.ld = ldx;
  q.W.ptr = Wg, q.W.ld = ldwg, q.W.layout = w_layout;
  q.W2.ptr = Wu, q.W2.ld = ldwu, q.W2.layout = w_layout;
  q.in_dtype = q.out_dtype = dtype;
  q.exact = precision_mode != GEMM_PREC_TF32;
  q.C = H, q.ldc = ldh;
  q.ep.act = activation;
  q.ep.pre = gate, q.ep.ld_pre = ld_gate;
  q.pre2 = up, q.ld_pre2 = ld_up;
  bool taken = false;
  st = fused(h, q, &taken, s);
  if (taken) return st;
  // Both products in fp32 (into gate and up themselves when those are fp32), then h.
  const bool keep32 = gate && dtype == GEMM_F32;
  Problem PG = G, PU = U;
  PG.out_dtype = PU.out_dtype = GEMM_F32;
  if (keep32) {
    PG.C = gate, PG.ldc = ld_gate, PU.C = up, PU.ldc = ld_up;
  } else {
    PG.ldc = PU.ldc = round_up(F, 4);
    Carve carve;
    const size_t off = carve.take(M * PG.ldc, 4);
    const size_t off_u = carve.take(M * PG.ldc, 4);
    st = reserve(h, h->ff, carve.bytes, s);
    if (st != GEMM_OK) return st;
    PG.C = static_cast<char *>(h->ff.ptr) + off;
    PU.C = static_cast<char *>(h->ff.ptr) + off_u;
  }
  st = product(h, PG, s);
  if (st == GEMM_OK) st = product(h, PU, s);
  if (st != GEMM_OK) return st;
  const float *g32 = static_cast<const float *>(PG.C), *u32 = static_cast<const float *>(PU.C);
  if (gate && !keep32) {
    const ff::Epilogue none;
    st = launched(h, ff::epilogue_rows_launch(g32, PG.ldc, gate, ld_gate, dtype, none, M, F, s), "gate store");
    if (st == GEMM_OK)
      st = launched(h, ff::epilogue_rows_launch(u32, PU.ldc, up, ld_up, dtype, none, M, F, s), "up store");
    if (st != GEMM_OK) return st;
  }
  return launched(h, ff::gated_rows_launch(g32, PG.ldc, u32, PU.ldc, H, ldh, dtype, activation, M, F, s),
                  "gated launch");
}

GEMM_API gemm_status_t gemm_run_gated_backward(
    gemm_handle_t h, int64_t M, int64_t F, int64_t K, const void *dH, int64_t lddh,
    const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, const void *X, int64_t ldx,
    const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu, void *dX, int64_t lddx, void *dWg,
    int64_t lddwg, void *dWu, int64_t lddwu, gemm_dtype_t dtype, gemm_precision_t precision_mode,
    gemm_layout_t w_layout, gemm_activation_t activation, void *cuda_stream) {
  if (!h || M < 0 || F < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(dtype) || !valid_act(activation) || !valid_layout(w_layout) ||
      precision_mode < GEMM_PREC_DEFAULT || precision_mode > GEMM_PREC_F16_ACC)
    return GEMM_ERR_INVALID_ARG;
  const bool weights = dWg || dWu;
  if (bad_matrix(dH, M, F, lddh, GEMM_ROW_MAJOR) || bad_matrix(gate, M, F, ld_gate, GEMM_ROW_MAJOR) ||
      bad_matrix(up, M, F, ld_up, GEMM_ROW_MAJOR) ||
      (weights && bad_matrix(X, M, K, ldx, GEMM_ROW_MAJOR)) ||
      (dWg && bad_matrix(dWg, K, F, lddwg, w_layout)) ||
      (dWu && bad_matrix(dWu, K, F, lddwu, w_layout)) ||
      (dX && (bad_matrix(dX, M, K, lddx, GEMM_ROW_MAJOR) || bad_matrix(Wg, K, F, ldwg, w_layout) ||
              bad_matrix(Wu, K, F, ldwu, w_layout))))
    return GEMM_ERR_INVALID_ARG;
  if (precision_mode == GEMM_PREC_F16_ACC ||
      (dtype != GEMM_F32 && precision_mode != GEMM_PREC_DEFAULT))
    return GEMM_ERR_UNSUPPORTED;
  if (M > INT32_MAX || 2 * F > INT32_MAX || K > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
  const int es = esize_of(dtype);
  for (const void *p : {dH, gate, up, X, Wg, Wu, static_cast<const void *>(dX),
                        static_cast<const void *>(dWg), static_cast<const void *>(dWu)})
    if (misaligned(p, es)) return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(dX, M, K, lddx, GEMM_ROW_MAJOR, es),
                       matrix_span(dWg, K, F, lddwg, w_layout, es),
                       matrix_span(dWu, K, F, lddwu, w_layout, es)};
  const Span ins[] = {matrix_span(dH, M, F, lddh, GEMM_ROW_MAJOR, es),
                      matrix_span(gate, M, F, ld_gate, GEMM_ROW_MAJOR, es),
                      matrix_span(up, M, F, ld_up, GEMM_ROW_MAJOR, es),
                      weights ? matrix_span(X, M, K, ldx, GEMM_ROW_MAJOR, es) : Span{},
                      dX ? matrix_span(Wg, K, F, ldwg, w_layout, es) : Span{},
                      dX ? matrix_span(Wu, K, F, ldwu, w_layout, es) : Span{}};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  if (!dX && !weights) return GEMM_OK;
  DeviceGuard guard(h->device);
  if (!guard.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  // dg | du side by side, so that one product can take both
  const int64_t Fp = round_up(F, 16 / es), ldd = 2 * Fp;
  const int64_t ld32 = round_up(K, 4);
  const bool make_dx = dX && M > 0 && K > 0;
  Carve carve;
  const size_t d_off = carve.take(M * ldd, es);
  ff::FusedProduct q;  // dX = dg Wg^T + du Wu^T in one accumulator
  q.M = M, q.N = K, q.K = q.K2 = F;
  q.X.ld = q.X2.ld = ldd;
  // (addresses in the handle's buffer once it is sized; 256-byte aligned, so never staged)
  q.W.ptr = Wg, q.W.ld = ldwg, q.W2.ptr = Wu, q.W2.ld = ldwu;
  q.W.layout = q.W2.layout = flip(w_layout);
  q.in_dtype = q.out_dtype = dtype;
  q.C = dX, q.ldc = lddx;
  const bool taken = make_dx && ff::plan_fused(h, &q, &carve);
  const size_t x_off = make_dx && !taken ? carve.take(M * ld32, 4) : 0;
  const size_t x2_off = make_dx && !taken ? carve.take(M * ld32, 4) : 0;
  gemm_status_t st = reserve(h, h->ff, carve.bytes, s);
  if (st != GEMM_OK) return st;
  char *buf = static_cast<char *>(h->ff.ptr);
  char *dg = buf + d_off, *du = dg + Fp * es;
  if (M > 0 && F > 0) {
    st = launched(h, ff::gated_slopes_launch(dH, lddh, gate, ld_gate, up, ld_up, dg, ldd, du, ldd,
                                             dtype, activation, M, F, s),
                  "gated backward launch");
    if (st != GEMM_OK) return st;
  }
  bool summed = false;
  if (taken) {
    q.X.ptr = dg, q.X2.ptr = du;
    st = ff::run_fused(h, q, buf, s);
    if (st != GEMM_OK) return st;
  } else if (make_dx) {
    // two products in fp32, added and rounded once; in one step with the second product where
    // an fp32 kernel takes it
    if (dtype == GEMM_F32) {
      ff::FusedProduct r;
      r.M = M, r.N = K, r.K = F;
      r.X.ptr = du, r.X.ld = ldd;
      r.W.ptr = Wu, r.W.ld = ldwu, r.W.layout = flip(w_layout);
      r.in_dtype = r.out_dtype = GEMM_F32;
      r.exact = precision_mode != GEMM_PREC_TF32;
      r.C = dX, r.ldc = lddx;
      r.ep.residual = dX, r.ep.ld_residual = lddx;
      Carve none;
      if (ff::plan_fused(h, &r, &none)) {
        st = product(h, Problem{M, K, F, dg, ldd, Wg, ldwg, dX, lddx, dtype, dtype, precision_mode,
                                GEMM_ROW_MAJOR, flip(w_layout)}, s);
        if (st == GEMM_OK) st = ff::run_fused(h, r, nullptr, s);
        if (st != GEMM_OK) return st;
        summed = true;
      }
    }
  }
  if (!taken && make_dx && !summed) {
    float *x32 = reinterpret_cast<float *>(buf + x_off), *x2 = reinterpret_cast<float *>(buf + x2_off);
    st = product(h, Problem{M, K, F, dg, ldd, Wg, ldwg, x32, ld32, dtype, GEMM_F32, precision_mode,
                            GEMM_ROW_MAJOR, flip(w_layout)}, s);
    if (st == GEMM_OK)
      st = product(h, Problem{M, K, F, du, ldd, Wu, ldwu, x2, ld32, dtype, GEMM_F32, precision_mode,
                              GEMM_ROW_MAJOR, flip(w_layout)}, s);
    if (st == GEMM_OK)
      st = launched(h, ff::add_rows_launch(x32, ld32, x2, ld32, dX, lddx, dtype, M, K, s), "sum of products");
    if (st != GEMM_OK) return st;
  }
  // Gradients that adjoin in memory are one product with both halves of dg | du.
  if (dWg && dWu && Fp == F && w_layout == GEMM_COL_MAJOR && lddwg == lddwu &&
      static_cast<char *>(dWu) - static_cast<char *>(dWg) == F * lddwg * es)
    return operand_gradients(h, M, 2 * F, K, dg, ldd, X, ldx, GEMM_ROW_MAJOR, nullptr, 0, w_layout,
                             nullptr, 0, dWg, lddwg, dtype, precision_mode, s);
  for (int i = 0; i < 2 && st == GEMM_OK; ++i) {
    void *dW = i ? dWu : dWg;
    if (!dW) continue;
    st = operand_gradients(h, M, F, K, i ? du : dg, ldd, X, ldx, GEMM_ROW_MAJOR, nullptr, 0, w_layout,
                           nullptr, 0, dW, i ? lddwu : lddwg, dtype, precision_mode, s);
  }
  return st;
}

GEMM_API gemm_status_t gemm_layer_norm(gemm_handle_t h, int64_t M, int64_t N, const void *X,
                                       int64_t ldx, const void *weight, const void *bias, void *Y,
                                       int64_t ldy, float *mean, float *rstd, float eps,
                                       gemm_dtype_t in_dtype, gemm_dtype_t param_dtype,
                                       gemm_dtype_t out_dtype, void *cuda_stream) {
  if (!h || M < 0 || N < 0) return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || !valid_dtype(param_dtype))
    return GEMM_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  if (bad_matrix(X, M, N, ldx, GEMM_ROW_MAJOR) || bad_matrix(Y, M, N, ldy, GEMM_ROW_MAJOR))
    return GEMM_ERR_INVALID_ARG;
  if (M > INT32_MAX || N > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
  const int is = esize_of(in_dtype), os = esize_of(out_dtype), ps = esize_of(param_dtype);
  if (misaligned(X, is) || misaligned(Y, os) || misaligned(weight, ps) || misaligned(bias, ps) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return GEMM_ERR_ALIGNMENT;
  const bool in_place = X == Y && ldx == ldy && in_dtype == out_dtype;
  const Span outs[] = {matrix_span(Y, M, N, ldy, GEMM_ROW_MAJOR, os), vector_span(mean, M, 4),
                       vector_span(rstd, M, 4)};
  const Span x = matrix_span(X, M, N, ldx, GEMM_ROW_MAJOR, is);
  const Span ins[] = {in_place ? Span{} : x, vector_span(weight, N, ps), vector_span(bias, N, ps)};
  if (!disjoint(outs, ins) || outs[1].meets(x) || outs[2].meets(x)) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  return launched(h, ff::layer_norm_launch(X, ldx, in_dtype, weight, bias, param_dtype, Y, ldy,
                                           out_dtype, mean, rstd, eps, M, N, h->sm_count,
                                           static_cast<cudaStream_t>(cuda_stream)),
                  "layer norm launch");
}

GEMM_API gemm_status_t gemm_layer_norm_backward(gemm_handle_t h, int64_t M, int64_t N,
                                                const void *dY, int64_t lddy, const void *X,
                                                int64_t ldx, const void *weight,
                                                const float *mean, const float *rstd, void *dX,
                                                int64_t lddx, void *dweight, void *dbias,
                                                gemm_dtype_t in_dtype, gemm_dtype_t param_dtype,
                                                gemm_dtype_t out_dtype, void *cuda_stream) {
  if (!h || M < 0 || N < 0) return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || !valid_dtype(param_dtype))
    return GEMM_ERR_INVALID_ARG;
  if (N == 0) return GEMM_OK;
  if (bad_matrix(dY, M, N, lddy, GEMM_ROW_MAJOR) || bad_matrix(X, M, N, ldx, GEMM_ROW_MAJOR) ||
      (dX && bad_matrix(dX, M, N, lddx, GEMM_ROW_MAJOR)) || (M > 0 && (!mean || !rstd)))
    return GEMM_ERR_INVALID_ARG;
  if (M > INT32_MAX || N > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
  const int is = esize_of(in_dtype), os = esize_of(out_dtype), ps = esize_of(param_dtype);
  if (misaligned(dY, os) || misaligned(X, is) || misaligned(weight, ps) || misaligned(mean, 4) ||
      misaligned(rstd, 4) || misaligned(dX, is) || misaligned(dweight, ps) || misaligned(dbias, ps))
    return GEMM_ERR_ALIGNMENT;
  const Span outs[] = {matrix_span(dX, M, N, lddx, GEMM_ROW_MAJOR, is), vector_span(dweight, N, ps),
                       vector_span(dbias, N, ps)};
  const Span ins[] = {matrix_span(dY, M, N, lddy, GEMM_ROW_MAJOR, os),
                      matrix_span(X, M, N, ldx, GEMM_ROW_MAJOR, is), vector_span(weight, N, ps),
                      vector_span(mean, M, 4), vector_span(rstd, M, 4)};
  if (!disjoint(outs, ins)) return GEMM_ERR_INVALID_ARG;
  if (!dX && !dweight && !dbias) return GEMM_OK;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  gemm_status_t st = reserve(
      h, h->ff, ff::layer_norm_backward_bytes(M, N, in_dtype == out_dtype, h->sm_count), s);
  if (st != GEMM_OK) return st;
  int launches = 0;
  const cudaError_t e = ff::layer_norm_backward_launch(
      dY, lddy, out_dtype, X, ldx, in_dtype, weight, param_dtype, mean, rstd, dX, lddx, dweight,
      dbias, h->ff.ptr, M, N, h->sm_count, &launches, s);
  return launched(h, e, "layer norm backward launch", launches);
}

}  // extern "C"
