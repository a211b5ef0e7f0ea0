// expert_launch.h -- host side of the experts' products: operands as the caller stores them and as
// the kernels read them, copies of those TMA cannot address, tensor maps, launch. Internal to the
// library.
#pragma once

#include "api_internal.h"
#include "expert_kernels.h"
#include "ff_launch.h"

namespace gemm_gb300 {
namespace ff {

// Rows (rows x cols, row-major) or the experts' matrices (`count` of `lines` x `len`, as stored),
// copied into the handle's buffer first where TMA cannot read them in place.
struct ExpertOperand {
  const void *ptr = nullptr;
  int64_t lines = 0, len = 0, ld = 0;
  int64_t count = 1, stride = 0;
  bool staged = false;
  size_t offset = 0;
  // Decides whether it is copied, and where.
  void plan(Carve *carve);
  // Makes the copy in `buf`; ptr, ld and stride are then the copy's. With offsets only matrices of
  // experts that have rows are copied (the others are not read).
  gemm_status_t stage(gemm_handle_t h, char *buf, cudaStream_t s, const int32_t *offsets = nullptr);
};

// The experts' weights as a call gives them: K x N of each expert in `layout`.
ExpertOperand expert_weights(const void *W, int64_t ld, int64_t stride, int64_t experts, int64_t K,
                             int64_t N, int layout);
ExpertOperand expert_rows(const void *X, int64_t ld, int64_t rows, int64_t cols);

struct ExpertProduct {
  bool gated = false;
  int64_t experts = 0, rows = 0, N = 0, K = 0;
  const int32_t *offsets = nullptr;
  ExpertOperand X, X2, W, W2;  // X2, W2: the second of a sum (W2: of the gated pair)
  bool second = false;         // a sum of two products of one K
  bool w_mn = false;           // weights stored with the output features inside
  int dtype = GEMM_BF16, act = GEMM_ACT_NONE;
  void *C = nullptr;
  int64_t ldc = 0;
  void *pre = nullptr, *pre2 = nullptr;
  int64_t ld_pre = 0, ld_pre2 = 0;
};
gemm_status_t run_expert(gemm_handle_t h, const ExpertProduct &q, cudaStream_t s);

// D[e] = sum over e's rows of A[r]^T B[r], stored MA x NB.
struct ExpertGrad {
  int64_t experts = 0, rows = 0;
  const int32_t *offsets = nullptr;
  ExpertOperand A, B;
  int dtype = GEMM_BF16;
  void *D = nullptr;
  int64_t ldd = 0, stride_d = 0;
};
gemm_status_t run_expert_grad(gemm_handle_t h, const ExpertGrad &q, cudaStream_t s);

// The same two products in fp32, operands as the caller stores them.
gemm_status_t run_expert_f32(gemm_handle_t h, const ExpertProduct &q, bool add, cudaStream_t s);
gemm_status_t run_expert_grad_f32(gemm_handle_t h, const ExpertGrad &q, cudaStream_t s);

// Whether the tiles of a call can be numbered in 32 bits.
bool expert_tiles_fit(int64_t experts, int64_t rows, int64_t N, int64_t K);

}  // namespace ff
}  // namespace gemm_gb300
