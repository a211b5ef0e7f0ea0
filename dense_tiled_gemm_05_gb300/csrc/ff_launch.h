// ff_launch.h -- the fused products: what a call asks for, whether and how
// the tensor-core kernels take it, and the launch. Internal to the library.
#pragma once

#include "api_internal.h"
#include "ff_kernels.h"

namespace gemm_gb300 {
namespace ff {

// The handle's feed-forward buffer, cut into 256-byte aligned pieces.
struct Carve {
  size_t bytes = 0;
  size_t take(int64_t n, int es) {
    const size_t off = bytes;
    bytes += static_cast<size_t>(api::round_up(n * es, 256));
    return off;
  }
};

// One operand as the caller stores it and, after plan_fused, as the kernel reads it: X is
// read row-major (K-major), W in its own layout. An operand TMA cannot address (or a
// column-major X) is copied into the handle's buffer first.
struct FusedOperand {
  const void *ptr = nullptr;
  int64_t ld = 0;
  int layout = GEMM_ROW_MAJOR;
  bool staged = false, transpose = false;
  size_t offset = 0;
  int64_t staged_ld = 0;
};

struct FusedProduct {
  bool gated = false;
  int64_t M = 0, N = 0;
  int64_t K = 0, K2 = 0;   // K2 > 0: the sum of two products
  FusedOperand X, W, X2, W2;  // gated: W2 is the second projection, K2 is 0
  int in_dtype = GEMM_BF16, out_dtype = GEMM_BF16;
  bool exact = true;       // fp32 inputs at full precision (else tf32)
  void *C = nullptr;
  int64_t ldc = 0;
  Epilogue ep;             // gated: act, pre and ld_pre only
  void *pre2 = nullptr;
  int64_t ld_pre2 = 0;
  // plan
  enum Kind { kToken, kTile, kFew, kPair } kind = kPair;
  int tile_size = 64;      // tile kernel
  int tile_splits = 1;
  int k_warps = 1;         // token kernel
  bool vector = false;     // token kernel: 16-byte accesses
  FewParams few_params{};
  double few_cost = 0.0;   // few-token kernel's estimate, SM cycles
  int64_t tiles_m = 0, tiles_n = 0;
};

// Whether the fused kernels take the product (16-bit types, and fp32 for a few tokens or
// small exact products); fills the plan and adds the staged copies to `carve`. False: a type, size or option they do not
// handle.
bool plan_fused(gemm_handle_t h, FusedProduct *q, Carve *carve);
// `buf`: the buffer the offsets of plan_fused refer to.
gemm_status_t run_fused(gemm_handle_t h, const FusedProduct &q, char *buf, cudaStream_t s);

}  // namespace ff
}  // namespace gemm_gb300
