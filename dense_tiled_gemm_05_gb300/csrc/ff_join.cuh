// ff_join.cuh -- the end of a product tile whose K a cluster's CTAs share: every CTA's fp32
// partial waits in its own shared memory, and after a cluster barrier each CTA sums a share of
// the outputs over all of them, in rank order, applies the epilogue and stores.
#pragma once

#include "activation.cuh"
#include "ff_kernels.h"
#include "ptx.cuh"

namespace gemm_gb300 {
namespace ff {

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ void store4(T *row, int64_t n, int64_t N, bool vec, const float (&v)[4]) {
  if (vec)
    store_piece<T, 4, true>(row, n, N, v);
  else
    store_piece<T, 4, false>(row, n, N, v);
}

// Epilogue of four consecutive columns n.. of row m from their fp32 sums. vec: the outputs and
// the residual allow four-element accesses.
template <typename TO, bool GATED, bool FAST>
__device__ __forceinline__ void finish4(const FusedParams &p, bool vec, int64_t m, int64_t n,
                                        float (&a)[4], float (&b)[4]) {
  if (GATED) {
    if (p.pre) {
      store4(static_cast<TO *>(p.pre) + m * p.ld_pre, n, p.N, vec, a);
      store4(static_cast<TO *>(p.pre2) + m * p.ld_pre2, n, p.N, vec, b);
    }
    activate_all<FAST>(a, p.act);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] *= b[i];
  } else {
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) a[i] += load_any(p.bias, p.bias_dtype, n + i);
    }
    if (p.pre) store4(static_cast<TO *>(p.pre) + m * p.ld_pre, n, p.N, vec, a);
    activate_all<FAST>(a, p.act);
    if (p.residual) {
      const TO *r = static_cast<const TO *>(p.residual) + m * p.ld_residual;
      if (vec)
        load_piece<TO, 4, true>(r, n, p.N, b);
      else
        load_piece<TO, 4, false>(r, n, p.N, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] += b[i];
    }
  }
  store4(static_cast<TO *>(p.C) + m * p.ldc, n, p.N, vec, a);
}

template <bool GATED, bool FAST>
__device__ __forceinline__ void finish4_any(const FusedParams &p, bool vec, int64_t m, int64_t n,
                                            float (&a)[4], float (&b)[4]) {
  if (p.out_dtype == GEMM_BF16)
    finish4<__nv_bfloat16, GATED, FAST>(p, vec, m, n, a, b);
  else if (p.out_dtype == GEMM_F16)
    finish4<__half, GATED, FAST>(p, vec, m, n, a, b);
  else
    finish4<float, GATED, FAST>(p, vec, m, n, a, b);
}

// Partials: [row][COLS] fp32 at shared address `base` of each of the `splits` CTAs (gated: the
// second product's `plane` floats on), for `rows` rows from m0 and columns from n0. A thread's
// items of four columns are BATCH at a time: all their partials are on the way before the first
// sum, or each would wait for the other SMs' shared memory in turn.
template <bool GATED, bool FAST, int COLS, int THREADS, int BATCH>
__device__ __forceinline__ void join_partials(const FusedParams &p, bool vec, uint32_t base,
                                              int plane, int rows, int splits, int rank,
                                              int64_t m0, int64_t n0) {
  const int items = rows * (COLS / 4), stride = splits * THREADS;
  for (int i0 = rank * THREADS + static_cast<int>(threadIdx.x); i0 < items; i0 += BATCH * stride) {
    float a[BATCH][4], b[BATCH][4];
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[j][i] = b[j][i] = 0.0f;
#pragma unroll 2
    for (int q = 0; q < splits; ++q) {
      float4 v[BATCH], w[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int i = min(i0 + j * stride, items - 1);
        const uint32_t at = mapa_shared(base + static_cast<uint32_t>(i) * 16, static_cast<uint32_t>(q));
        v[j] = ld_cluster_f4(at);
        if (GATED) w[j] = ld_cluster_f4(at + plane * static_cast<uint32_t>(sizeof(float)));
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        a[j][0] += v[j].x, a[j][1] += v[j].y, a[j][2] += v[j].z, a[j][3] += v[j].w;
        if (GATED) b[j][0] += w[j].x, b[j][1] += w[j].y, b[j][2] += w[j].z, b[j][3] += w[j].w;
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = i0 + j * stride;
      const int64_t n = n0 + i % (COLS / 4) * 4;
      if (i < items && n < p.N)
        finish4_any<GATED, FAST>(p, vec, m0 + i / (COLS / 4), n, a[j], b[j]);
    }
  }
}

}  // namespace ff
}  // namespace gemm_gb300
