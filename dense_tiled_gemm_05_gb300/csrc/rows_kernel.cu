// rows_kernel.cu -- the feed-forward operators' elementwise and column-sum kernels:
//
//   y  = act(z + bias) + residual          (after a product kept in fp32)
//   h  = act(g) * u
//   dg = dh u act'(g),  du = dh act(g)
//   dz = dy act'(pre),  dbias_j = sum_i dz_ij
//
// All are bound by the bytes they read and write. A warp covers 256 columns of a row, eight a
// lane: consecutive ones in 16-byte accesses where the rows allow it, else every 32nd, so that
// a request's lanes are neighbours. A CTA's eight warps take eight rows at a time. Sums over rows are kept in fp32
// registers over a band of rows and joined over the CTA's warps in shared memory, then over
// the bands in a second kernel, always in the same order.
#include "activation.cuh"
#include "ff_internal.h"
#include "pdl.h"
#include "ptx.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 32 * VEC;       // columns a CTA

bool aligned16(const void *p, int64_t ld, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0);
}
int esize(int dt) { return dt == GEMM_F32 ? 4 : 2; }

// A warp walks rows of its 256 columns, so that the loads of several rows overlap: about ten
// CTAs for every one of 152 SMs, whatever the matrix (more rows a warp and fewer CTAs start
// unevenly, one row a warp spends its time starting CTAs: 8192 x 8192 slopes took 191 us).
dim3 rows_grid(int64_t M, int64_t N) {
  const int64_t gx = (N + kCols - 1) / kCols;
  const int64_t all = (M + kWarps - 1) / kWarps;
  int64_t gy = (1520 + gx - 1) / gx;
  if (gy > all) gy = all;
  if (gy > 65535) gy = 65535;
  return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
}

#define FF_ROWS(i, M)                                                                     \
  for (int64_t i = static_cast<int64_t>(blockIdx.y) * kWarps + threadIdx.x / 32; i < M;   \
       i += static_cast<int64_t>(gridDim.y) * kWarps)

template <bool VECTOR>
__device__ __forceinline__ Columns<32, VECTOR> my_columns(int64_t N) {
  return {static_cast<int64_t>(blockIdx.x) * kCols, N, static_cast<int>(threadIdx.x % 32)};
}

// (z and y may be one buffer: a lane reads its columns before it writes them)
template <typename TO, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    epilogue_rows_kernel(const float *z, int64_t ldz, TO *y, int64_t ldy, const Epilogue ep,
                         int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const auto cols = my_columns<VECTOR>(N);
  if (!cols.in(0)) return;
  float b[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    b[i] = ep.bias && cols.in(i) ? load_any(ep.bias, ep.bias_dtype, cols.at(i)) : 0.0f;
#pragma unroll 2
  FF_ROWS(i, M) {
    float v[VEC], r[VEC];
    cols.load_f32(z + i * ldz, v);
    if (ep.residual) cols.load_f32(static_cast<const TO *>(ep.residual) + i * ep.ld_residual, r);
#pragma unroll
    for (int c = 0; c < VEC; ++c) v[c] += b[c];
    if (ep.pre) cols.store(static_cast<TO *>(ep.pre) + i * ep.ld_pre, v);
    activate_all<false>(v, ep.act);
    if (ep.residual) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) v[c] += r[c];
    }
    cols.store(y + i * ldy, v);
  }
}

template <typename TO, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    gated_rows_kernel(const float *__restrict__ g, int64_t ldg, const float *__restrict__ u,
                      int64_t ldu, TO *__restrict__ h, int64_t ldh, int act, int64_t M, int64_t F) {
  grid_dependency_wait();
  grid_launch_dependents();
  const auto cols = my_columns<VECTOR>(F);
  if (!cols.in(0)) return;
#pragma unroll 2
  FF_ROWS(i, M) {
    float a[VEC], b[VEC];
    cols.load_f32(g + i * ldg, a);
    cols.load_f32(u + i * ldu, b);
    activate_all<false>(a, act);
#pragma unroll
    for (int c = 0; c < VEC; ++c) a[c] *= b[c];
    cols.store(h + i * ldh, a);
  }
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    gated_slopes_kernel(const T *__restrict__ dh, int64_t lddh, const T *__restrict__ g,
                        int64_t ldg, const T *__restrict__ u, int64_t ldu, T *__restrict__ dg,
                        int64_t lddg, T *__restrict__ du, int64_t lddu, int act, int64_t M,
                        int64_t F) {
  grid_dependency_wait();
  grid_launch_dependents();
  const auto cols = my_columns<VECTOR>(F);
  if (!cols.in(0)) return;
#pragma unroll 2
  FF_ROWS(i, M) {
    float vh[VEC], vg[VEC], vu[VEC], a[VEC], d[VEC];
    cols.load_f32(dh + i * lddh, vh);
    cols.load_f32(g + i * ldg, vg);
    cols.load_f32(u + i * ldu, vu);
    activate_slope_all<sizeof(T) == 2>(vg, act, a, d);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      vg[c] = vh[c] * vu[c] * d[c];
      vu[c] = vh[c] * a[c];
    }
    // (16-bit types: the rounding that makes dg and du operands of the tensor cores)
    cols.store(dg + i * lddg, vg);
    cols.store(du + i * lddu, vu);
  }
}

template <typename TO, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    add_rows_kernel(const float *a, int64_t lda, const float *__restrict__ b, int64_t ldb, TO *y,
                    int64_t ldy, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const auto cols = my_columns<VECTOR>(N);
  if (!cols.in(0)) return;
#pragma unroll 2
  FF_ROWS(i, M) {
    float v[VEC], w[VEC];
    cols.load_f32(a + i * lda, v);
    cols.load_f32(b + i * ldb, w);
#pragma unroll
    for (int c = 0; c < VEC; ++c) v[c] += w[c];
    cols.store(y + i * ldy, v);
  }
}

// dz = dy act'(pre), and the sums of dz (before it is rounded) over the CTA's band of rows.
template <typename TG, typename TZ, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    epilogue_slopes_kernel(const TG *__restrict__ dy, int64_t lddy, const TG *__restrict__ pre,
                           int64_t ld_pre, int act, TZ *__restrict__ dz, int64_t lddz,
                           float *__restrict__ partials, int64_t M, int64_t N, int64_t band) {
  __shared__ float red[kWarps][kCols];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  grid_dependency_wait();
  grid_launch_dependents();
  const auto cols = my_columns<VECTOR>(N);
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * band;
  const int64_t hi = lo + band < M ? lo + band : M;
  float sum[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) sum[c] = 0.0f;
  if (cols.in(0)) {
#pragma unroll 2
    for (int64_t i = lo + warp; i < hi; i += kWarps) {
      float v[VEC];
      cols.load_f32(dy + i * lddy, v);
      if (pre) {
        float z[VEC], a[VEC], d[VEC];
        cols.load_f32(pre + i * ld_pre, z);
        activate_slope_all<sizeof(TZ) == 2>(z, act, a, d);
#pragma unroll
        for (int c = 0; c < VEC; ++c) v[c] *= d[c];
      }
#pragma unroll
      for (int c = 0; c < VEC; ++c) sum[c] += v[c];
      if (dz) cols.store(dz + i * lddz, v);
    }
  }
  if (!partials) return;
#pragma unroll
  for (int c = 0; c < VEC; ++c) red[warp][c * 32 + lane] = sum[c];
  __syncthreads();
  // thread t joins piece t / 32 of lane t % 32 over the warps
  const int c = threadIdx.x / 32;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += red[w][c * 32 + lane];
  if (cols.in(c)) partials[static_cast<int64_t>(blockIdx.y) * N + cols.at(c)] = s;
}

// 32 columns a CTA; its 32 warps take every 32nd band, eight loads in flight each, and are
// joined in their order. (Eight warps took 9 us for 304 bands of 4096 columns.)
__global__ void __launch_bounds__(1024)
    column_finish_kernel(const float *__restrict__ partials, int64_t bands, int sums,
                         void *out0, void *out1, int dtype, int64_t N) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int which = blockIdx.y;
  grid_dependency_wait();
  grid_launch_dependents();
  float s = 0.0f;
  if (j < N) {
#pragma unroll 8
    for (int64_t b = warp; b < bands; b += 32) s += partials[(b * sums + which) * N + j];
  }
  red[warp][lane] = s;
  __syncthreads();
  // warp w joins column w of the CTA: lane l holds warp l's sum
  s = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && col < N) store_any(which ? out1 : out0, dtype, col, s);
}

}  // namespace

// Bands of rows: enough CTAs for about four on every SM, at least 64 rows each so that the
// partial sums stay a small part of what is read.
int64_t column_bands(int64_t M, int64_t N, int sm_count) {
  const int64_t cols = (N + kCols - 1) / kCols;
  int64_t bands = (4 * static_cast<int64_t>(sm_count > 0 ? sm_count : 1) + cols - 1) / cols;
  const int64_t most = (M + 63) / 64;
  if (bands > most) bands = most;
  if (bands > 65535) bands = 65535;
  return bands < 1 ? 1 : bands;
}

cudaError_t epilogue_rows_launch(const float *z, int64_t ldz, void *y, int64_t ldy, int out_dtype,
                                 const Epilogue &ep, int64_t M, int64_t N, cudaStream_t s) {
  const int os = esize(out_dtype);
  const bool vec = N % VEC == 0 && aligned16(z, ldz, 4) && aligned16(y, ldy, os) &&
                   aligned16(ep.residual, ep.ld_residual, os) && aligned16(ep.pre, ep.ld_pre, os);
  const dim3 grid = rows_grid(M, N);
  FF_TYPED(out_dtype, T, {
    if (vec)
      launch_pdl(epilogue_rows_kernel<T, true>, grid, kThreads, 0, s, z, ldz, static_cast<T *>(y), ldy, ep, M, N);
    else
      launch_pdl(epilogue_rows_kernel<T, false>, grid, kThreads, 0, s, z, ldz, static_cast<T *>(y), ldy, ep, M, N);
  })
  return cudaGetLastError();
}

cudaError_t gated_rows_launch(const float *g, int64_t ldg, const float *u, int64_t ldu, void *h,
                              int64_t ldh, int out_dtype, int act, int64_t M, int64_t F,
                              cudaStream_t s) {
  const bool vec = F % VEC == 0 && aligned16(g, ldg, 4) && aligned16(u, ldu, 4) && aligned16(h, ldh, esize(out_dtype));
  const dim3 grid = rows_grid(M, F);
  FF_TYPED(out_dtype, T, {
    if (vec)
      launch_pdl(gated_rows_kernel<T, true>, grid, kThreads, 0, s, g, ldg, u, ldu, static_cast<T *>(h), ldh, act, M, F);
    else
      launch_pdl(gated_rows_kernel<T, false>, grid, kThreads, 0, s, g, ldg, u, ldu, static_cast<T *>(h), ldh, act, M, F);
  })
  return cudaGetLastError();
}

cudaError_t gated_slopes_launch(const void *dh, int64_t lddh, const void *g, int64_t ldg,
                                const void *u, int64_t ldu, void *dg, int64_t lddg, void *du,
                                int64_t lddu, int dtype, int act, int64_t M, int64_t F,
                                cudaStream_t s) {
  const int es = esize(dtype);
  const bool vec = F % VEC == 0 && aligned16(dh, lddh, es) && aligned16(g, ldg, es) && aligned16(u, ldu, es) &&
                   aligned16(dg, lddg, es) && aligned16(du, lddu, es);
  const dim3 grid = rows_grid(M, F);
  FF_TYPED(dtype, T, {
    auto kernel = vec ? gated_slopes_kernel<T, true> : gated_slopes_kernel<T, false>;
    launch_pdl(kernel, grid, kThreads, 0, s, static_cast<const T *>(dh), lddh, static_cast<const T *>(g), ldg,
                                     static_cast<const T *>(u), ldu, static_cast<T *>(dg), lddg,
                                     static_cast<T *>(du), lddu, act, M, F);
  })
  return cudaGetLastError();
}

cudaError_t add_rows_launch(const float *a, int64_t lda, const float *b, int64_t ldb, void *y,
                            int64_t ldy, int out_dtype, int64_t M, int64_t N, cudaStream_t s) {
  const bool vec = N % VEC == 0 && aligned16(a, lda, 4) && aligned16(b, ldb, 4) && aligned16(y, ldy, esize(out_dtype));
  const dim3 grid = rows_grid(M, N);
  FF_TYPED(out_dtype, T, {
    if (vec)
      launch_pdl(add_rows_kernel<T, true>, grid, kThreads, 0, s, a, lda, b, ldb, static_cast<T *>(y), ldy, M, N);
    else
      launch_pdl(add_rows_kernel<T, false>, grid, kThreads, 0, s, a, lda, b, ldb, static_cast<T *>(y), ldy, M, N);
  })
  return cudaGetLastError();
}

cudaError_t column_finish_launch(const float *partials, int64_t bands, int sums, void *out0,
                                 void *out1, int dtype, int64_t N, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((N + 31) / 32), static_cast<unsigned>(out1 ? 2 : 1));
  launch_pdl(column_finish_kernel, grid, 1024, 0, s, partials, bands, sums, out0, out1, dtype, N);
  return cudaGetLastError();
}

cudaError_t epilogue_slopes_launch(const void *dy, int64_t lddy, const void *pre, int64_t ld_pre,
                                   int grad_dtype, int act, void *dz, int64_t lddz, int dz_dtype,
                                   void *dbias, int bias_dtype, float *partials, int64_t M,
                                   int64_t N, int sm_count, cudaStream_t s) {
  const int gs = esize(grad_dtype);
  const bool vec = N % VEC == 0 && aligned16(dy, lddy, gs) && aligned16(pre, ld_pre, gs) &&
                   aligned16(dz, lddz, esize(dz_dtype));
  const int64_t bands = column_bands(M, N, sm_count);
  const int64_t band = (M + bands - 1) / bands;
  const dim3 grid(static_cast<unsigned>((N + kCols - 1) / kCols), static_cast<unsigned>(bands));
  float *part = dbias ? partials : nullptr;
  FF_TYPED(grad_dtype, TG, {
    FF_TYPED(dz_dtype, TZ, {
      auto kernel = vec ? epilogue_slopes_kernel<TG, TZ, true> : epilogue_slopes_kernel<TG, TZ, false>;
      launch_pdl(kernel, grid, kThreads, 0, s, static_cast<const TG *>(dy), lddy, static_cast<const TG *>(pre),
                                       ld_pre, act, static_cast<TZ *>(dz), lddz, part, M, N, band);
    })
  })
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dbias) return e;
  return column_finish_launch(partials, bands, 1, dbias, nullptr, bias_dtype, N, s);
}

}  // namespace ff
}  // namespace gemm_gb300
