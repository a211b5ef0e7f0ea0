// row_piece.cuh -- a warp's 256 columns of a row, eight a lane: consecutive ones in 16-byte accesses
// where rows allow it (VECTOR: they start on 16-byte boundaries and are a multiple of eight long),
// else every 32nd, so that a request's lanes are neighbours. As Columns in activation.cuh, with one
// address and one bound a lane, which leaves the loops over elements immediate offsets and 32-bit
// comparisons (8000 rows of 3001 bf16 through dropout: 26.5 us, 32 with Columns).
#pragma once

#include "activation.cuh"

namespace gemm_gb300 {
namespace ff {

template <bool VECTOR>
struct RowPiece {
  int64_t first;  // this lane's first column
  int left;       // columns from there to the row's end
  __device__ __forceinline__ RowPiece(int64_t c0, int64_t n, int lane)
      : first(c0 + (VECTOR ? lane * VEC : lane)), left(static_cast<int>(n - first)) {}

  template <typename E>
  __device__ __forceinline__ void load(const E *row, E (&e)[VEC]) const {
    const E *p = row + first;
    if (VECTOR) {
#pragma unroll
      for (int w = 0; w < VEC * static_cast<int>(sizeof(E)) / 16; ++w)
        reinterpret_cast<uint4 *>(e)[w] = left > 0 ? reinterpret_cast<const uint4 *>(p)[w] : uint4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = 32 * i < left ? p[32 * i] : from_f32<E>(0.0f);
    }
  }
  // The bits as they are (E: any type of their size).
  template <typename E>
  __device__ __forceinline__ void store_raw(E *row, const E (&e)[VEC]) const {
    E *p = row + first;
    if (VECTOR) {
      if (left > 0) {
#pragma unroll
        for (int w = 0; w < VEC * static_cast<int>(sizeof(E)) / 16; ++w)
          reinterpret_cast<uint4 *>(p)[w] = reinterpret_cast<const uint4 *>(e)[w];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (32 * i < left) p[32 * i] = e[i];
    }
  }
  template <typename E>
  __device__ __forceinline__ void load_f32(const E *row, float (&v)[VEC]) const {
    alignas(16) E e[VEC];
    load(row, e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
  }
  template <typename E>
  __device__ __forceinline__ void store(E *row, const float (&v)[VEC]) const {
    alignas(16) E e[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_f32<E>(v[i]);
    store_raw(row, e);
  }
};

}  // namespace ff
}  // namespace gemm_gb300
