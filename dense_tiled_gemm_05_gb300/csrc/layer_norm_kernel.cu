// layer_norm_kernel.cu -- layer norm of the rows of an M x N matrix and its backward pass:
//
//   mean_i = sum_j x_ij / N,  var_i = sum_j (x_ij - mean_i)^2 / N,  rstd_i = 1 / sqrt(var_i + eps)
//   y_ij   = (x_ij - mean_i) rstd_i w_j + b_j
//
//   xh = (x - mean) rstd,  v = dy w
//   dx_ij  = rstd_i (v_ij - mean_j(v) - xh_ij mean_j(v xh))
//   dw_j   = sum_i dy_ij xh_ij,   db_j = sum_i dy_ij
//
// Both are bound by HBM: the forward pass has to read x and write y, the backward pass to
// read x and dy and write dx. A row is held in the registers of a group of threads, so that
// each of these moves once; the variance is that of the centred values (a second reduction
// over registers, not E[x^2] - mean^2, which loses all digits when |mean| >> std). Sums and
// statistics are fp32.
#include "activation.cuh"
#include "ff_internal.h"

namespace gemm_gb300 {
namespace ff {
namespace {

int esize(int dt) { return dt == GEMM_F32 ? 4 : 2; }
bool aligned16(const void *p, int64_t ld, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Barrier of the T threads of group g (T a multiple of 32; ids 1.. of the CTA's 16).
template <int T>
__device__ __forceinline__ void group_sync(int g) {
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(T) : "memory");
}

// Sum over the T threads of a group; every thread gets it. `red`: T / 32 floats of the group's
// own; consecutive calls alternate between two such arrays, so that one barrier a call is
// enough (a thread writes an array again only after the barrier of the call in between).
template <int T>
__device__ __forceinline__ float group_sum(float v, float *red, int g) {
  v = warp_sum(v);
  if (T == 32) return v;
  const int warp = (threadIdx.x % T) / 32;
  if (threadIdx.x % 32 == 0) red[warp] = v;
  group_sync<T>(g);
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) s += red[w];
  return s;
}

// Two sums at once (`red`: 2 T / 32 floats).
template <int T>
__device__ __forceinline__ void group_sum2(float &a, float &b, float *red, int g) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (T == 32) return;
  const int warp = (threadIdx.x % T) / 32;
  if (threadIdx.x % 32 == 0) {
    red[2 * warp] = a;
    red[2 * warp + 1] = b;
  }
  group_sync<T>(g);
  a = b = 0.0f;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    a += red[2 * w];
    b += red[2 * w + 1];
  }
}

// Threads of a CTA: one group of T, or as many groups of T as make up 128 threads.
template <int T>
constexpr int kCtaThreads = T < 128 ? 128 : T;

// ------------------------------------------------------------------------- forward

// A group of T threads a row; a thread holds CH chunks of VEC consecutive columns, chunk c of
// thread t being columns (c T + t) VEC ... .
template <typename TI, typename TO, int T, int CH, bool VECTOR>
__global__ void __launch_bounds__(kCtaThreads<T>)
    norm_rows_kernel(const TI *x, int64_t ldx, const void *weight, const void *bias,
                     int param_dtype, TO *y, int64_t ldy, float *mean_out, float *rstd_out,
                     float eps, int64_t M, int64_t N) {
  constexpr int VEC = 16 / sizeof(TI);
  constexpr int G = kCtaThreads<T> / T;
  __shared__ float red[G][2][T / 32];
  const int g = threadIdx.x / T, t = threadIdx.x % T;
  const float n = static_cast<float>(N);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * G + g; row < M;
       row += static_cast<int64_t>(gridDim.x) * G) {
    float v[CH][VEC];
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      load_piece<TI, VEC, VECTOR>(x + row * ldx, (static_cast<int64_t>(c) * T + t) * VEC, N, v[c]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += v[c][i];
    }
    const float mean = group_sum<T>(s, red[g][0], g) / n;
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[c][i] -= mean;
        if ((static_cast<int64_t>(c) * T + t) * VEC + i < N) q = fmaf(v[c][i], v[c][i], q);
      }
    const float rstd = rsqrtf(group_sum<T>(q, red[g][1], g) / n + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t j0 = (static_cast<int64_t>(c) * T + t) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const bool in = j0 + i < N;
        const float w = weight && in ? load_any(weight, param_dtype, j0 + i) : 1.0f;
        const float b = bias && in ? load_any(bias, param_dtype, j0 + i) : 0.0f;
        v[c][i] = fmaf(v[c][i] * rstd, w, b);
      }
      store_piece<TO, VEC, VECTOR>(y + row * ldy, j0, N, v[c]);
    }
    if (t == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// Rows too long for a CTA's registers: three passes over the row, the later two mostly from
// L2 (the rows in flight fit in it).
template <typename TI, typename TO, bool VECTOR>
__global__ void __launch_bounds__(512)
    norm_long_rows_kernel(const TI *x, int64_t ldx, const void *weight, const void *bias,
                          int param_dtype, TO *y, int64_t ldy, float *mean_out, float *rstd_out,
                          float eps, int64_t M, int64_t N) {
  constexpr int T = 512, VEC = 16 / sizeof(TI);
  __shared__ float red[2][T / 32];
  const float n = static_cast<float>(N);
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const TI *xr = x + row * ldx;
    float v[VEC], s = 0.0f;
    for (int64_t j0 = threadIdx.x * VEC; j0 < N; j0 += T * VEC) {
      load_piece<TI, VEC, VECTOR>(xr, j0, N, v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += v[i];
    }
    const float mean = group_sum<T>(s, red[0], 0) / n;
    float q = 0.0f;
    for (int64_t j0 = threadIdx.x * VEC; j0 < N; j0 += T * VEC) {
      load_piece<TI, VEC, VECTOR>(xr, j0, N, v);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (j0 + i < N) q = fmaf(v[i] - mean, v[i] - mean, q);
    }
    const float rstd = rsqrtf(group_sum<T>(q, red[1], 0) / n + eps);
    for (int64_t j0 = threadIdx.x * VEC; j0 < N; j0 += T * VEC) {
      load_piece<TI, VEC, VECTOR>(xr, j0, N, v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const bool in = j0 + i < N;
        const float w = weight && in ? load_any(weight, param_dtype, j0 + i) : 1.0f;
        const float b = bias && in ? load_any(bias, param_dtype, j0 + i) : 0.0f;
        v[i] = fmaf((v[i] - mean) * rstd, w, b);
      }
      store_piece<TO, VEC, VECTOR>(y + row * ldy, j0, N, v);
    }
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// ------------------------------------------------------------------------ backward

// mean_j(v) and mean_j(v xh) of each row, by a warp a row.
template <typename TG, typename TI, bool VECTOR>
__global__ void __launch_bounds__(256)
    norm_row_means_kernel(const TG *__restrict__ dy, int64_t lddy, const TI *__restrict__ x,
                          int64_t ldx, const void *weight, int param_dtype,
                          const float *__restrict__ mean, const float *__restrict__ rstd,
                          float2 *__restrict__ means, int64_t M, int64_t N) {
  constexpr int VEC = 8;
  const float n = static_cast<float>(N);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; row < M;
       row += static_cast<int64_t>(gridDim.x) * 8) {
    const float mu = mean[row], r = rstd[row];
    float a = 0.0f, b = 0.0f;
    for (int64_t j0 = (threadIdx.x % 32) * VEC; j0 < N; j0 += 32 * VEC) {
      float vx[VEC], vd[VEC];
      load_piece<TI, VEC, VECTOR>(x + row * ldx, j0, N, vx);
      load_piece<TG, VEC, VECTOR>(dy + row * lddy, j0, N, vd);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float w = weight && j0 + i < N ? load_any(weight, param_dtype, j0 + i) : 1.0f;
        const float v = vd[i] * w;  // 0 past the row's end: dy reads as 0 there
        a += v;
        b = fmaf(v, (vx[i] - mu) * r, b);
      }
    }
    a = warp_sum(a);
    b = warp_sum(b);
    if (threadIdx.x % 32 == 0) means[row] = make_float2(a / n, b / n);
  }
}

// dx and the sums of dy xh and dy over a band of rows, from the rows' means: a warp covers
// 256 columns, a CTA's eight warps eight rows at a time.
template <typename TG, typename TI, bool VECTOR>
__global__ void __launch_bounds__(256)
    norm_columns_kernel(const TG *__restrict__ dy, int64_t lddy, const TI *__restrict__ x,
                        int64_t ldx, const void *weight, int param_dtype,
                        const float *__restrict__ mean, const float *__restrict__ rstd,
                        const float2 *__restrict__ means, TI *__restrict__ dx, int64_t lddx,
                        float *__restrict__ partials, int64_t M, int64_t N, int64_t band) {
  constexpr int VEC = 8;
  __shared__ float red[2][8][32 * VEC];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t j0 = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * VEC;
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * band;
  const int64_t hi = lo + band < M ? lo + band : M;
  float w[VEC], dw[VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    w[i] = weight && j0 + i < N ? load_any(weight, param_dtype, j0 + i) : 1.0f;
    dw[i] = db[i] = 0.0f;
  }
  if (j0 < N) {
#pragma unroll 2
    for (int64_t row = lo + warp; row < hi; row += 8) {
      float vx[VEC], vd[VEC];
      load_piece<TI, VEC, VECTOR>(x + row * ldx, j0, N, vx);
      load_piece<TG, VEC, VECTOR>(dy + row * lddy, j0, N, vd);
      const float mu = mean[row], r = rstd[row];
      const float2 m = means[row];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float xh = (vx[i] - mu) * r;
        dw[i] = fmaf(vd[i], xh, dw[i]);
        db[i] += vd[i];
        vx[i] = r * (fmaf(vd[i], w[i], -m.x) - xh * m.y);
      }
      if (dx) store_piece<TI, VEC, VECTOR>(dx + row * lddx, j0, N, vx);
    }
  }
  if (!partials) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    red[0][warp][i * 32 + lane] = dw[i];
    red[1][warp][i * 32 + lane] = db[i];
  }
  __syncthreads();
  const int i = threadIdx.x / 32;
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    a += red[0][k][i * 32 + lane];
    b += red[1][k][i * 32 + lane];
  }
  if (j0 + i < N) {
    partials[(static_cast<int64_t>(blockIdx.y) * 2) * N + j0 + i] = a;
    partials[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * N + j0 + i] = b;
  }
}

// --------------------------------------------------------------------- dispatch

struct NormArgs {
  const void *x;
  int64_t ldx;
  const void *weight, *bias;
  int param_dtype;
  void *y;
  int64_t ldy;
  float *mean, *rstd;
  float eps;
  int64_t M, N;
  bool vec;
  int sm_count;
  cudaStream_t s;
};

template <typename TI, typename TO, int T, int CH>
void launch_rows(const NormArgs &a) {
  constexpr int G = kCtaThreads<T> / T;
  const int64_t ctas = (a.M + G - 1) / G;
  const int64_t cap = static_cast<int64_t>(a.sm_count > 0 ? a.sm_count : 1) * 64;
  const int grid = static_cast<int>(ctas < cap ? ctas : cap);
  auto kernel = a.vec ? norm_rows_kernel<TI, TO, T, CH, true> : norm_rows_kernel<TI, TO, T, CH, false>;
  kernel<<<grid, kCtaThreads<T>, 0, a.s>>>(static_cast<const TI *>(a.x), a.ldx, a.weight, a.bias,
                                             a.param_dtype, static_cast<TO *>(a.y), a.ldy, a.mean,
                                             a.rstd, a.eps, a.M, a.N);
}

// Threads a row: the fewest (32 .. 1024) that hold it at 16 values a thread, then 1024 at 32.
template <typename TI, typename TO>
void dispatch_rows(const NormArgs &a) {
  constexpr int VEC = 16 / sizeof(TI), C16 = 16 / VEC, C32 = 32 / VEC;
  const int64_t pieces = (a.N + VEC - 1) / VEC;
  if (pieces <= 32 * C16) return launch_rows<TI, TO, 32, C16>(a);
  if (pieces <= 64 * C16) return launch_rows<TI, TO, 64, C16>(a);
  if (pieces <= 128 * C16) return launch_rows<TI, TO, 128, C16>(a);
  if (pieces <= 256 * C16) return launch_rows<TI, TO, 256, C16>(a);
  if (pieces <= 512 * C16) return launch_rows<TI, TO, 512, C16>(a);
  if (pieces <= 1024 * C16) return launch_rows<TI, TO, 1024, C16>(a);
  if (pieces <= 1024 * C32) return launch_rows<TI, TO, 1024, C32>(a);
  const int64_t cap = static_cast<int64_t>(a.sm_count > 0 ? a.sm_count : 1) * 64;
  const int grid = static_cast<int>(a.M < cap ? a.M : cap);
  auto kernel = a.vec ? norm_long_rows_kernel<TI, TO, true> : norm_long_rows_kernel<TI, TO, false>;
  kernel<<<grid, 512, 0, a.s>>>(static_cast<const TI *>(a.x), a.ldx, a.weight, a.bias,
                                a.param_dtype, static_cast<TO *>(a.y), a.ldy, a.mean, a.rstd, a.eps,
                                a.M, a.N);
}

}  // namespace

cudaError_t layer_norm_launch(const void *x, int64_t ldx, int in_dtype, const void *weight,
                              const void *bias, int param_dtype, void *y, int64_t ldy,
                              int out_dtype, float *mean, float *rstd, float eps, int64_t M,
                              int64_t N, int sm_count, cudaStream_t s) {
  const bool vec = aligned16(x, ldx, esize(in_dtype)) && aligned16(y, ldy, esize(out_dtype));
  const NormArgs a{x, ldx, weight, bias, param_dtype, y, ldy, mean, rstd, eps, M, N, vec, sm_count, s};
  FF_TYPED(in_dtype, TI, { FF_TYPED(out_dtype, TO, { dispatch_rows<TI, TO>(a); }) })
  return cudaGetLastError();
}

size_t layer_norm_backward_bytes(int64_t M, int64_t N, int sm_count) {
  return static_cast<size_t>((M * sizeof(float2) + 255) / 256 * 256) +
         column_partials_bytes(M, N, 2, sm_count);
}

cudaError_t layer_norm_backward_launch(const void *dy, int64_t lddy, int grad_dtype, const void *x,
                                       int64_t ldx, int in_dtype, const void *weight,
                                       int param_dtype, const float *mean, const float *rstd,
                                       void *dx, int64_t lddx, void *dweight, void *dbias,
                                       void *workspace, int64_t M, int64_t N, int sm_count,
                                       int *launches, cudaStream_t s) {
  const int is = esize(in_dtype);
  const bool vec = aligned16(dy, lddy, esize(grad_dtype)) && aligned16(x, ldx, is) &&
                   aligned16(dx, lddx, is);
  float2 *means = static_cast<float2 *>(workspace);
  float *partials = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                              (M * sizeof(float2) + 255) / 256 * 256);
  const int64_t bands = column_bands(M, N, sm_count);
  const int64_t band = (M + bands - 1) / bands;
  const int64_t ctas = (M + 7) / 8, cap = static_cast<int64_t>(sm_count > 0 ? sm_count : 1) * 32;
  const dim3 grid(static_cast<unsigned>((N + 255) / 256), static_cast<unsigned>(bands));
  float *part = dweight || dbias ? partials : nullptr;
  FF_TYPED(grad_dtype, TG, {
    FF_TYPED(in_dtype, TI, {
      if (M > 0) {
        auto k1 = vec ? norm_row_means_kernel<TG, TI, true> : norm_row_means_kernel<TG, TI, false>;
        k1<<<static_cast<unsigned>(ctas < cap ? ctas : cap), 256, 0, s>>>(
            static_cast<const TG *>(dy), lddy, static_cast<const TI *>(x), ldx, weight, param_dtype,
            mean, rstd, means, M, N);
        ++*launches;
      }
      auto k2 = vec ? norm_columns_kernel<TG, TI, true> : norm_columns_kernel<TG, TI, false>;
      k2<<<grid, 256, 0, s>>>(static_cast<const TG *>(dy), lddy, static_cast<const TI *>(x), ldx,
                              weight, param_dtype, mean, rstd, means, static_cast<TI *>(dx), lddx,
                              part, M, N, band);
      ++*launches;
    })
  })
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !part) return e;
  // (column_finish's first output is the first sum: with no dweight, dbias is the second)
  ++*launches;
  if (dweight) return column_finish_launch(partials, bands, 2, dweight, dbias, param_dtype, N, s);
  return column_finish_launch(partials + N, bands, 2, dbias, nullptr, param_dtype, N, s);
}

}  // namespace ff
}  // namespace gemm_gb300
