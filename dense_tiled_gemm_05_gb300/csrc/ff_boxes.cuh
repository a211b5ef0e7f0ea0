// ff_boxes.cuh -- from TMEM to the 32-row, 128-byte-wide boxes that the pair kernels' epilogues
// store by TMA.
#pragma once

#include "tc_common.cuh"

namespace gemm_gb300 {
namespace ff {

using tc::pack2;

// COLS consecutive accumulator columns of this lane's row, as fp32. By whole warps, whose lanes
// may come from rows past M or from a store that one of them issued.
template <int COLS>
__device__ __forceinline__ void read_columns(uint32_t taddr, float (&v)[COLS]) {
  __syncwarp();
  uint32_t r[COLS / 32][32];
#pragma unroll
  for (int h = 0; h < COLS / 32; ++h) tmem_ld_32x32b_x32(taddr + h * 32, r[h]);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < COLS; ++i) v[i] = __uint_as_float(r[i / 32][i % 32]);
}

// One row of a 32-row, 128-byte-wide box (128-byte swizzle): v rounded to OUT.
template <int OUT, int COLS>
__device__ __forceinline__ void write_box_row(uint32_t row_addr, int lane, const float (&v)[COLS]) {
  constexpr int PER = OUT == GEMM_F32 ? 4 : 8;  // elements in 16 bytes
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = OUT == GEMM_F32 ? __float_as_uint(v[ch * PER + i])
                             : pack2<OUT>(__float_as_uint(v[ch * PER + 2 * i]),
                                          __float_as_uint(v[ch * PER + 2 * i + 1]));
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + ((ch ^ (lane & 7)) << 4)),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
}

}  // namespace ff
}  // namespace gemm_gb300
