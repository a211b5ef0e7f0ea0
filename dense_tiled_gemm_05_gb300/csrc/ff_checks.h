// ff_checks.h -- argument checks shared by the C entries of the feed-forward operators and of
// the operators of experts: the spans of a call's buffers, which outputs have to keep off, and
// alignment. Host only; internal to the library.
#pragma once

#include "api_internal.h"

namespace gemm_gb300 {
namespace ff {

inline bool valid_act(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SIGMOID; }

// A buffer of a call: the bytes it spans and, for a matrix, its line pitch and the bytes of a
// line, to keep outputs off inputs and each other. Several matrices also have the pitch from one to
// the next and the bytes of one (block_pitch 0: one matrix).
struct Span {
  uintptr_t lo = 0, hi = 0;  // empty: lo == hi
  uintptr_t pitch = 0, line = 0;
  uintptr_t block_pitch = 0, block = 0;
  bool meets(const Span &o) const {
    if (!(lo < o.hi && o.lo < hi)) return false;
    // column ranges of one wider matrix, or parts of matrices that follow one another at one pitch,
    // share a span, but no element
    return !(apart(o, pitch, line, o.pitch, o.line) || apart(o, pitch, line, o.block_pitch, o.block) ||
             apart(o, block_pitch, block, o.pitch, o.line) ||
             apart(o, block_pitch, block, o.block_pitch, o.block));
  }

 private:
  // Whether `len` bytes at lo + i * step and `len_o` bytes at o.lo + j * step are apart for all i, j.
  bool apart(const Span &o, uintptr_t step, uintptr_t len, uintptr_t step_o, uintptr_t len_o) const {
    if (step == 0 || step != step_o) return false;
    const uintptr_t d = (lo < o.lo ? o.lo - lo : step - (lo - o.lo) % step) % step;
    return d >= len && d + len_o <= step;
  }
};

inline Span matrix_span(const void *p, int64_t rows, int64_t cols, int64_t ld, int layout, int es) {
  Span s;
  if (!p || rows <= 0 || cols <= 0) return s;
  api::span_of(p, rows, cols, ld, layout, es, &s.lo, &s.hi);
  s.pitch = static_cast<uintptr_t>(ld * es);
  s.line = static_cast<uintptr_t>((layout == GEMM_ROW_MAJOR ? cols : rows) * es);
  return s;
}
inline Span vector_span(const void *p, int64_t n, int es) {
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

inline bool misaligned(const void *p, int es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

// A row-major or column-major operand of a call that is used: pointer and leading dimension.
inline bool bad_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int layout) {
  if (rows == 0 || cols == 0) return false;
  return !p || ld < (layout == GEMM_ROW_MAJOR ? cols : rows);
}

inline gemm_status_t launched(gemm_handle_t h, cudaError_t e, const char *what, int n = 1) {
  if (e != cudaSuccess) return api::cuda_fail(e, what);
  h->launches += static_cast<uint64_t>(n);
  return GEMM_OK;
}

}  // namespace ff
}  // namespace gemm_gb300
