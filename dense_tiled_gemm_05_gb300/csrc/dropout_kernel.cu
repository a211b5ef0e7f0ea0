// dropout_kernel.cu -- y = x * mask / keep + residual, the mask made from a counter:
//
// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel Random Numbers: As Easy as 1,
// 2, 3", SC 2011) maps the counter (column / 8, row, offset) under the key (seed) to four 32-bit
// words, which are eight 16-bit numbers, the low half of a word first. Element (row, column)
// takes number column % 8 and is kept where that is not below round(65536 p). The kept share of
// the 65536 numbers is exact; the scale is its inverse rounded to fp32 (2^-24 of it at most). The
// same key gives the same mask whatever the strides, so the backward pass
// makes it again and nothing is stored.
//
// Bound by the bytes of x, residual and y: sixteen bits an element cost one generator call (20
// wide multiplications) for eight elements; with 32 bits an element that would be two. A lane
// takes eight neighbouring columns, its own generator block. Rows that do not allow 16-byte
// accesses are read and written every 32nd column a lane, the numbers handed over through
// shared memory. (16384 x 4096 bf16 with a residual: 62.6 us, 6.4 TB/s.)
#include <algorithm>

#include "activation.cuh"
#include "expert_internal.h"
#include "pdl.h"
#include "ptx.cuh"
#include "row_piece.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 32 * VEC;

__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                               uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return uint4{c0, c1, c2, c3};
}

// (y may be x or the residual: a lane reads its columns of a row before it writes them)
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(const T *x, int64_t ldx, const T *residual, int64_t ldr, T *y, int64_t ldy,
                   uint32_t threshold, float scale, const uint64_t *__restrict__ key, int64_t M,
                   int64_t N) {
  __shared__ uint4 shared[VECTOR ? 1 : kThreads];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint64_t seed = key[0], offset = key[1];
  const RowPiece<VECTOR> cols(static_cast<int64_t>(blockIdx.x) * kCols, N, lane);
  const uint32_t block = static_cast<uint32_t>(blockIdx.x) * 32 + lane;
  const uint32_t row_step = gridDim.y * kWarps;
#pragma unroll 2
  for (uint32_t i = blockIdx.y * kWarps + warp; i < M; i += row_step) {
    float v[VEC], r[VEC];
    cols.load_f32(x + static_cast<int64_t>(i) * ldx, v);
    if (residual) cols.load_f32(residual + static_cast<int64_t>(i) * ldr, r);
    const uint4 words = philox4x32_10(block, i, static_cast<uint32_t>(offset),
                                      static_cast<uint32_t>(offset >> 32), static_cast<uint32_t>(seed),
                                      static_cast<uint32_t>(seed >> 32));
    uint32_t number[VEC];
    if (VECTOR) {
      const uint32_t q[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
      for (int c = 0; c < VEC; ++c) number[c] = c % 2 ? q[c / 2] >> 16 : q[c / 2] & 0xFFFFu;
    } else {
      __syncwarp();  // the previous row's numbers have been read
      shared[threadIdx.x] = words;
      __syncwarp();
      const uint16_t *mine = reinterpret_cast<const uint16_t *>(shared + warp * 32);
#pragma unroll
      for (int c = 0; c < VEC; ++c) number[c] = mine[c * 32 + lane];
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      v[c] = number[c] >= threshold ? v[c] * scale : 0.0f;
      if (residual) v[c] += r[c];
    }
    cols.store(y + static_cast<int64_t>(i) * ldy, v);
  }
}

}  // namespace

cudaError_t dropout_launch(const void *x, int64_t ldx, const void *residual, int64_t ldr, void *y,
                           int64_t ldy, int dtype, uint32_t threshold, float scale,
                           const uint64_t *key, int64_t M, int64_t N, cudaStream_t s) {
  const int es = dtype == GEMM_F32 ? 4 : 2;
  auto aligned = [&](const void *p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0);
  };
  const bool vector = aligned(x, ldx) && aligned(residual, ldr) && aligned(y, ldy) && N % VEC == 0;
  const int64_t gx = (N + kCols - 1) / kCols;
  const int64_t gy = std::min<int64_t>({(3040 + gx - 1) / gx, (M + kWarps - 1) / kWarps, 65535});
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  FF_TYPED(dtype, T, {
    auto go = [&](auto kernel) {
      launch_pdl(kernel, grid, kThreads, 0, s, static_cast<const T *>(x), ldx,
                 static_cast<const T *>(residual), ldr, static_cast<T *>(y), ldy, threshold, scale,
                 key, M, N);
    };
    vector ? go(dropout_kernel<T, true>) : go(dropout_kernel<T, false>);
  })
  return cudaGetLastError();
}

}  // namespace ff
}  // namespace gemm_gb300
