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

// Sums of one or two values over the T threads of a group; every thread gets them. `red`: K
// times T / 32 floats of the group's own; consecutive calls alternate between two such
// arrays, so that one barrier a call is enough (a thread writes an array again only after the
// barrier of the call in between).
template <int T, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float *red, int g) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (T == 32) return;
  constexpr int WARPS = T / 32;
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) red[k * WARPS + (threadIdx.x % T) / 32] = v[k];
  }
  group_sync<T>(g);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = red[k * WARPS + lane % WARPS];
#pragma unroll
    for (int o = WARPS / 2; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
}
template <int T>
__device__ __forceinline__ float group_sum(float v, float *red, int g) {
  float a[1] = {v};
  group_sum<T, 1>(a, red, g);
  return a[0];
}

// Threads of a CTA: one group of T, or as many groups of T as make up 256 threads; and the
// CTAs an SM is to hold of it (1024 threads at 64 registers).
template <int T>
struct Cta {
  static constexpr int THREADS = T < 256 ? 256 : T;
  static constexpr int GROUPS = THREADS / T;
  static constexpr int PER_SM = 1024 / THREADS;
};
constexpr int VEC = 8;  // columns a thread holds of a row (twice that in the widest form)

// A thread's eight columns among the 8 T from `first` on. VECTOR (rows start on 16-byte
// boundaries, and so do N and the parameters): eight consecutive ones, in 16-byte accesses.
// Otherwise every T-th one, so that the lanes of a warp read neighbours.
template <int T, bool VECTOR>
struct Columns {
  int64_t first, n;
  int t;
  __device__ __forceinline__ int64_t at(int i) const {
    return VECTOR ? first + t * VEC + i : first + i * T + t;
  }
  __device__ __forceinline__ bool in(int i) const { return at(VECTOR ? 0 : i) < n; }

  template <typename E>
  __device__ __forceinline__ void load(const E *row, E (&e)[VEC]) const {
    if (VECTOR) {
      constexpr int W = VEC * sizeof(E) / 16;
#pragma unroll
      for (int w = 0; w < W; ++w)
        reinterpret_cast<uint4 *>(e)[w] =
            in(0) ? reinterpret_cast<const uint4 *>(row + at(0))[w] : uint4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = in(i) ? row[at(i)] : from_f32<E>(0.0f);
    }
  }
  template <typename E>
  __device__ __forceinline__ void store(E *row, const float (&v)[VEC]) const {
    if (VECTOR) {
      constexpr int W = VEC * sizeof(E) / 16;
      alignas(16) E e[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = from_f32<E>(v[i]);
      if (in(0)) {
#pragma unroll
        for (int w = 0; w < W; ++w)
          reinterpret_cast<uint4 *>(row + at(0))[w] = reinterpret_cast<const uint4 *>(e)[w];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (in(i)) row[at(i)] = from_f32<E>(v[i]);
    }
  }
  __device__ __forceinline__ void store(void *base, int dtype, int64_t offset,
                                        const float (&v)[VEC]) const {
    FF_TYPED(dtype, E, { store(static_cast<E *>(base) + offset, v); })
  }
  // A parameter vector (1 or 0 for every column where there is none).
  __device__ __forceinline__ void params(const void *p, int dtype, float missing,
                                         float (&v)[VEC]) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = missing;
      return;
    }
    FF_TYPED(dtype, E, {
      alignas(16) E e[VEC];
      load(static_cast<const E *>(p), e);
      _Pragma("unroll") for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
    })
  }
};

// ------------------------------------------------------------------------- forward

// A group of T threads a row; piece c of thread t is columns (c T + t) 8 ... . The CTAs stay
// and walk the rows: with one piece a thread, weight and bias are read once into registers
// (read for every row they are four times the bytes of a bf16 row with fp32 parameters, from
// L2: 16384 x 4096 took 152 us that way), and the next row's loads are issued before the
// current row's reductions. Two pieces a thread leave no registers for the parameters.
template <typename TI, int T, int CH, bool VECTOR>
__global__ void __launch_bounds__(Cta<T>::THREADS, Cta<T>::PER_SM)
    norm_rows_kernel(const TI *x, int64_t ldx, const void *weight, const void *bias,
                     int param_dtype, void *y, int64_t ldy, int out_dtype, float *mean_out,
                     float *rstd_out, float eps, int64_t M, int64_t N) {
  constexpr int G = Cta<T>::GROUPS;
  __shared__ float red[G][2][T / 32];
  const int g = threadIdx.x / T, t = threadIdx.x % T;
  const float n = static_cast<float>(N);
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + g;
  if (row >= M) return;
  auto columns = [&](int c) { return Columns<T, VECTOR>{static_cast<int64_t>(c) * T * VEC, N, t}; };
  alignas(16) TI next[CH][VEC];
  float w[VEC], b[VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) columns(c).load(x + row * ldx, next[c]);
  if (CH == 1) {
    columns(0).params(weight, param_dtype, 1.0f, w);
    columns(0).params(bias, param_dtype, 0.0f, b);
  }
  for (; row < M; row += step) {
    float v[CH][VEC];
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[c][i] = to_f32(next[c][i]);
        s += v[c][i];
      }
    if (row + step < M) {
#pragma unroll
      for (int c = 0; c < CH; ++c) columns(c).load(x + (row + step) * ldx, next[c]);
    }
    const float mean = group_sum<T>(s, red[g][0], g) / n;
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[c][i] -= mean;
        if (columns(c).in(i)) q = fmaf(v[c][i], v[c][i], q);
      }
    const float rstd = rsqrtf(group_sum<T>(q, red[g][1], g) / n + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (CH > 1) {
        columns(c).params(weight, param_dtype, 1.0f, w);
        columns(c).params(bias, param_dtype, 0.0f, b);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[c][i] = fmaf(v[c][i] * rstd, w[i], b[i]);
      columns(c).store(y, out_dtype, row * ldy, v[c]);
    }
    if (t == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// Rows too long for a CTA's registers: three passes over the row, the later two mostly from
// L2 (the rows in flight fit in it).
template <typename TI, bool VECTOR>
__global__ void __launch_bounds__(512)
    norm_long_rows_kernel(const TI *x, int64_t ldx, const void *weight, const void *bias,
                          int param_dtype, void *y, int64_t ldy, int out_dtype, float *mean_out,
                          float *rstd_out, float eps, int64_t M, int64_t N) {
  constexpr int T = 512;
  __shared__ float red[2][T / 32];
  const float n = static_cast<float>(N);
  Columns<T, VECTOR> cols{0, N, static_cast<int>(threadIdx.x)};
  alignas(16) TI e[VEC];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const TI *xr = x + row * ldx;
    float s = 0.0f;
    for (cols.first = 0; cols.first < N; cols.first += T * VEC) {
      cols.load(xr, e);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += to_f32(e[i]);
    }
    const float mean = group_sum<T>(s, red[0], 0) / n;
    float q = 0.0f;
    for (cols.first = 0; cols.first < N; cols.first += T * VEC) {
      cols.load(xr, e);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = to_f32(e[i]) - mean;
        if (cols.in(i)) q = fmaf(d, d, q);
      }
    }
    const float rstd = rsqrtf(group_sum<T>(q, red[1], 0) / n + eps);
    for (cols.first = 0; cols.first < N; cols.first += T * VEC) {
      float v[VEC], w[VEC], b[VEC];
      cols.load(xr, e);
      cols.params(weight, param_dtype, 1.0f, w);
      cols.params(bias, param_dtype, 0.0f, b);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = fmaf((to_f32(e[i]) - mean) * rstd, w[i], b[i]);
      cols.store(y, out_dtype, row * ldy, v);
    }
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// ------------------------------------------------------------------------ backward

// One pass for rows a CTA's registers hold (8 columns a thread): a group of T threads a row,
// x and dy read once, with the next row's loads in flight during the current row's
// reduction, dx written, and the columns' sums of dy xh and dy kept in registers over all of
// the group's rows. The groups of a CTA join theirs at the end; column_finish adds the CTAs.
template <typename TI, int T, bool VECTOR>
__global__ void __launch_bounds__(Cta<T>::THREADS, Cta<T>::PER_SM)
    norm_backward_kernel(const TI *__restrict__ dy, int64_t lddy, const TI *__restrict__ x,
                         int64_t ldx, const void *weight, int param_dtype,
                         const float *__restrict__ mean, const float *__restrict__ rstd,
                         TI *__restrict__ dx, int64_t lddx, float *__restrict__ partials,
                         int32_t M, int64_t N) {
  constexpr int G = Cta<T>::GROUPS;
  __shared__ float red[G][2][2 * (T / 32)];
  __shared__ float join[G > 1 ? 2 : 1][G > 1 ? T * VEC : 1];
  __shared__ float4 ws[2][T];  // the weight: registers go to the columns' sums
  const int g = threadIdx.x / T, t = threadIdx.x % T;
  const Columns<T, VECTOR> cols{0, N, t};
  const int step = static_cast<int>(gridDim.x) * G;
  int row = static_cast<int>(blockIdx.x) * G + g;
  float dw[VEC], db[VEC];
  alignas(16) TI nx[VEC];
  alignas(16) TI nd[VEC];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](int i) {
    cols.load(x + i * ldx, nx);
    cols.load(dy + i * lddy, nd);
    nmu = mean[i];
    nr = rstd[i];
  };
  if (row < M) fetch(row);
  if (g == 0) {
    cols.params(weight, param_dtype, 1.0f, dw);
    ws[0][t] = make_float4(dw[0], dw[1], dw[2], dw[3]);
    ws[1][t] = make_float4(dw[4], dw[5], dw[6], dw[7]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < VEC; ++i) dw[i] = db[i] = 0.0f;
  int buf = 0;
  while (row < M) {
    const int next = M - row > step ? row + step : M;
    const float r = nr;
    float xh[VEC], d[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      xh[i] = (to_f32(nx[i]) - nmu) * r;
      d[i] = to_f32(nd[i]);
    }
    if (next < M) fetch(next);
    const float4 w0 = ws[0][t], w1 = ws[1][t];
    const float w[VEC] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {  // (dy reads as 0 past the row's end)
      dw[i] = fmaf(d[i], xh[i], dw[i]);
      db[i] += d[i];
      d[i] *= w[i];
      s[0] += d[i];
      s[1] = fmaf(d[i], xh[i], s[1]);
    }
    group_sum<T, 2>(s, red[g][buf], g);
    buf ^= 1;
    if (dx) {
      const float n = static_cast<float>(N);
      const float a = s[0] / n, b = s[1] / n;
#pragma unroll
      for (int i = 0; i < VEC; ++i) d[i] = r * (d[i] - a - xh[i] * b);
      cols.store(dx + row * lddx, d);
    }
    row = next;
  }
  if (!partials) return;
  if (G > 1) {  // in the groups' order
    for (int k = 0; k < G; ++k) {
      if (g == k) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          join[0][i * T + t] = k ? join[0][i * T + t] + dw[i] : dw[i];
          join[1][i * T + t] = k ? join[1][i * T + t] + db[i] : db[i];
        }
      }
      __syncthreads();
    }
    if (g != 0) return;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      dw[i] = join[0][i * T + t];
      db[i] = join[1][i * T + t];
    }
  }
  float *out = partials + static_cast<int64_t>(blockIdx.x) * 2 * N;
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (cols.in(i)) {
      out[cols.at(i)] = dw[i];
      out[N + cols.at(i)] = db[i];
    }
}

// Longer rows, and a dy of another type than x: the rows' means first, then columns.
// mean_j(v) and mean_j(v xh) of each row, by a warp a row.
template <typename TG, typename TI, bool VECTOR>
__global__ void __launch_bounds__(256)
    norm_row_means_kernel(const TG *__restrict__ dy, int64_t lddy, const TI *__restrict__ x,
                          int64_t ldx, const void *weight, int param_dtype,
                          const float *__restrict__ mean, const float *__restrict__ rstd,
                          float2 *__restrict__ means, int64_t M, int64_t N) {
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

//
// dx and the sums of dy xh and dy over a band of rows, from the rows' means: a warp covers
// 256 columns, a CTA's eight warps eight rows at a time.
template <typename TG, typename TI, bool VECTOR>
__global__ void __launch_bounds__(256)
    norm_columns_kernel(const TG *__restrict__ dy, int64_t lddy, const TI *__restrict__ x,
                        int64_t ldx, const void *weight, int param_dtype,
                        const float *__restrict__ mean, const float *__restrict__ rstd,
                        const float2 *__restrict__ means, TI *__restrict__ dx, int64_t lddx,
                        float *__restrict__ partials, int64_t M, int64_t N, int64_t band) {
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
  int out_dtype;
  float *mean, *rstd;
  float eps;
  int64_t M, N;
  bool vec;
  int sm_count;
  cudaStream_t s;
};

int grid_of(int64_t ctas, int sm_count, int per_sm) {
  const int64_t cap = static_cast<int64_t>(sm_count > 0 ? sm_count : 1) * per_sm;
  return static_cast<int>(ctas < 1 ? 1 : ctas < cap ? ctas : cap);
}

template <typename TI, int T, int CH>
void launch_rows(const NormArgs &a) {
  const int grid = grid_of((a.M + Cta<T>::GROUPS - 1) / Cta<T>::GROUPS, a.sm_count, Cta<T>::PER_SM);
  auto kernel = a.vec ? norm_rows_kernel<TI, T, CH, true> : norm_rows_kernel<TI, T, CH, false>;
  kernel<<<grid, Cta<T>::THREADS, 0, a.s>>>(static_cast<const TI *>(a.x), a.ldx, a.weight, a.bias,
                                            a.param_dtype, a.y, a.ldy, a.out_dtype, a.mean, a.rstd,
                                            a.eps, a.M, a.N);
}

// Threads that hold a row of N columns, eight each: 32 .. 1024.
int row_threads(int64_t N) {
  int t = 32;
  while (t < 1024 && t * VEC < N) t *= 2;
  return t;
}
constexpr int64_t kOnePassColumns = 1024 * VEC;

template <typename TI>
void dispatch_rows(const NormArgs &a) {
  if (a.N > 2 * kOnePassColumns) {
    auto kernel = a.vec ? norm_long_rows_kernel<TI, true> : norm_long_rows_kernel<TI, false>;
    kernel<<<grid_of(a.M, a.sm_count, 64), 512, 0, a.s>>>(
        static_cast<const TI *>(a.x), a.ldx, a.weight, a.bias, a.param_dtype, a.y, a.ldy,
        a.out_dtype, a.mean, a.rstd, a.eps, a.M, a.N);
    return;
  }
  if (a.N > kOnePassColumns) return launch_rows<TI, 1024, 2>(a);
  switch (row_threads(a.N)) {
    case 32: return launch_rows<TI, 32, 1>(a);
    case 64: return launch_rows<TI, 64, 1>(a);
    case 128: return launch_rows<TI, 128, 1>(a);
    case 256: return launch_rows<TI, 256, 1>(a);
    case 512: return launch_rows<TI, 512, 1>(a);
    default: return launch_rows<TI, 1024, 1>(a);
  }
}

}  // namespace

cudaError_t layer_norm_launch(const void *x, int64_t ldx, int in_dtype, const void *weight,
                              const void *bias, int param_dtype, void *y, int64_t ldy,
                              int out_dtype, float *mean, float *rstd, float eps, int64_t M,
                              int64_t N, int sm_count, cudaStream_t s) {
  const bool vec = aligned16(x, ldx, esize(in_dtype)) && aligned16(y, ldy, esize(out_dtype)) &&
                   aligned16(weight, 0, 4) && aligned16(bias, 0, 4) && N % VEC == 0;
  const NormArgs a{x, ldx, weight, bias, param_dtype, y, ldy, out_dtype, mean, rstd, eps, M, N,
                   vec, sm_count, s};
  FF_TYPED(in_dtype, TI, { dispatch_rows<TI>(a); })
  return cudaGetLastError();
}

namespace {

struct NormBackwardArgs {
  const void *dy;
  int64_t lddy;
  const void *x;
  int64_t ldx;
  const void *weight;
  int param_dtype;
  const float *mean, *rstd;
  void *dx;
  int64_t lddx;
  float *partials;
  int64_t M, N;
  bool vec;
  int grid;
  cudaStream_t s;
};

template <typename TI, int T>
void launch_backward(const NormBackwardArgs &a) {
  auto kernel = a.vec ? norm_backward_kernel<TI, T, true> : norm_backward_kernel<TI, T, false>;
  kernel<<<a.grid, Cta<T>::THREADS, 0, a.s>>>(
      static_cast<const TI *>(a.dy), a.lddy, static_cast<const TI *>(a.x), a.ldx, a.weight,
      a.param_dtype, a.mean, a.rstd, static_cast<TI *>(a.dx), a.lddx, a.partials,
      static_cast<int32_t>(a.M), a.N);
}

// Grid of the one-pass kernel: as many CTAs as stay on the SMs, or as have rows.
int backward_grid(int64_t M, int64_t N, int sm_count) {
  const int t = row_threads(N);
  const int64_t groups = t < 256 ? 256 / t : 1;
  return grid_of((M + groups - 1) / groups, sm_count, t < 256 ? 4 : 1024 / t);
}

}  // namespace

size_t layer_norm_backward_bytes(int64_t M, int64_t N, bool one_type, int sm_count) {
  if (N <= kOnePassColumns && one_type)
    return static_cast<size_t>(backward_grid(M, N, sm_count)) * 2 * N * sizeof(float);
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
  if (N <= kOnePassColumns && grad_dtype == in_dtype) {
    float *sums = static_cast<float *>(workspace);
    const int grid = backward_grid(M, N, sm_count);
    const NormBackwardArgs a{dy, lddy, x, ldx, weight, param_dtype, mean, rstd, dx, lddx,
                             dweight || dbias ? sums : nullptr, M, N,
                             vec && aligned16(weight, 0, 4) && N % VEC == 0, grid, s};
    FF_TYPED(in_dtype, TI, {
      switch (row_threads(N)) {
        case 32: launch_backward<TI, 32>(a); break;
        case 64: launch_backward<TI, 64>(a); break;
        case 128: launch_backward<TI, 128>(a); break;
        case 256: launch_backward<TI, 256>(a); break;
        case 512: launch_backward<TI, 512>(a); break;
        default: launch_backward<TI, 1024>(a); break;
      }
    })
    ++*launches;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partials) return e;
    ++*launches;
    if (dweight) return column_finish_launch(sums, grid, 2, dweight, dbias, param_dtype, N, s);
    return column_finish_launch(sums + N, grid, 2, dbias, nullptr, param_dtype, N, s);
  }
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
