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
#include "pdl.h"
#include "ptx.cuh"

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

// Sum of a value over the T threads of a group; every thread gets it. `red`: T / 32 floats of
// the group's own; consecutive calls alternate between two such arrays, so that one barrier a
// call is enough (a thread writes an array again only after the barrier of the call in between).
template <int T>
__device__ __forceinline__ float group_sum(float v, float *red, int g) {
  v = warp_sum(v);
  if (T == 32) return v;
  constexpr int WARPS = T / 32;
  const int lane = threadIdx.x % 32;
  if (lane == 0) red[(threadIdx.x % T) / 32] = v;
  group_sync<T>(g);
  v = red[lane % WARPS];
#pragma unroll
  for (int o = WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Two sums at once (T at most 512; `red`: twice as many floats): the lower half of a warp
// carries the first value's sum and the upper half the second's, in half the shuffles.
template <int T>
__device__ __forceinline__ float2 group_sum2(float a, float b, float *red, int g) {
  static_assert(T <= 512, "a half warp holds the warps' sums");
  constexpr int WARPS = T / 32;
  const int lane = threadIdx.x % 32;
  const bool low = lane < 16;
  float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (T > 32) {
    if (lane % 16 == 0) red[(low ? 0 : WARPS) + (threadIdx.x % T) / 32] = v;
    group_sync<T>(g);
    v = red[(low ? 0 : WARPS) + lane % WARPS];
#pragma unroll
    for (int o = WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}

// Threads of a CTA: one group of T threads, or as many as make up `AT_LEAST`.
template <int T, int AT_LEAST>
struct Cta {
  static constexpr int THREADS = T < AT_LEAST ? AT_LEAST : T;
  static constexpr int GROUPS = THREADS / T;
};

// s / n, correctly rounded but for the last bit, without a division's instructions: the
// quotient's residual corrects it (a row of equal values has exactly their mean).
__device__ __forceinline__ float mean_of(float s, float n, float inv_n) {
  const float q = s * inv_n, c = fmaf(-q, n, s);
  return c == c ? fmaf(c, inv_n, q) : q;  // (an infinite sum's mean is infinite)
}

// The rows ahead of the one a thread works on, in its own slots of shared memory: cp.async
// takes no registers, and a thread that reads only its own slots needs no barrier.
template <int WORDS, int STAGES, int THREADS>
struct RowRing {
  static constexpr int BYTES = WORDS * STAGES * THREADS * 16;
  uint4 *mem;
  __device__ __forceinline__ uint4 *slot(int stage, int w) const {
    return mem + (stage * WORDS + w) * THREADS + threadIdx.x;
  }
  __device__ __forceinline__ void copy(int stage, int w, const void *src) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(slot(stage, w)))),
                 "l"(src)
                 : "memory");
  }
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest of STAGES groups in flight has arrived.
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
  }
};

// ------------------------------------------------------------------------- forward

// Few rows (or rows that 16-byte accesses cannot read): T threads a row, eight columns each,
// so that a row's time is short; weight and bias in registers, the next row loaded during the
// current row's reductions.
template <typename TI, int T, bool VECTOR>
__global__ void __launch_bounds__(Cta<T, 256>::THREADS, 1024 / Cta<T, 256>::THREADS)
    norm_rows_kernel(const TI *x, int64_t ldx, const void *weight, const void *bias,
                     int param_dtype, void *y, int64_t ldy, int out_dtype, float *mean_out,
                     float *rstd_out, float eps, int64_t M, int64_t N) {
  constexpr int G = Cta<T, 256>::GROUPS;
  __shared__ float red[G][2][T / 32];
  const int g = threadIdx.x / T, t = threadIdx.x % T;
  const float n = static_cast<float>(N), inv_n = 1.0f / n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + g;
  if (row >= M) return;
  grid_dependency_wait();
  grid_launch_dependents();
  const Columns<T, VECTOR> cols{0, N, t};
  alignas(16) TI next[VEC];
  float w[VEC], b[VEC];
  cols.load(x + row * ldx, next);
  cols.params(weight, param_dtype, 1.0f, w);
  cols.params(bias, param_dtype, 0.0f, b);
  for (; row < M; row += step) {
    float v[VEC];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[i] = to_f32(next[i]);
      s += v[i];
    }
    if (row + step < M) cols.load(x + (row + step) * ldx, next);
    const float mean = mean_of(group_sum<T>(s, red[g][0], g), n, inv_n);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[i] -= mean;
      if (cols.in(i)) q = fmaf(v[i], v[i], q);
    }
    const float rstd = rsqrtf(mean_of(group_sum<T>(q, red[g][1], g), n, inv_n) + eps);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = fmaf(v[i] * rstd, w[i], b[i]);
    cols.store(y, out_dtype, row * ldy, v);
    if (t == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// Many rows: 32 columns a thread, four pieces of eight, (c T + t) 8 ... for piece c. The
// reductions' instructions are per thread, so wide threads make the kernel wait for memory
// and not for issue slots (8 columns a thread issued 0.7 instructions a cycle and scheduler
// and moved 4.5 TB/s on 16384 x 4096 bf16). The CTAs stay and walk the rows: weight and bias
// wait in shared memory in fp32 (from L2 they are four times the bytes of a bf16 row), the
// next row in the ring.
constexpr int kWidePieces = 4;
template <typename TI, int T>
struct WideNorm {
  using C = Cta<T, 512>;
  static constexpr int WORDS = kWidePieces * VEC * static_cast<int>(sizeof(TI)) / 16;
  static constexpr int STAGES = WORDS > 4 ? 1 : 2;
  using Ring = RowRing<WORDS, STAGES, C::THREADS>;
  static constexpr int COLUMNS = T * kWidePieces * VEC;
  static constexpr int SMEM = Ring::BYTES + 2 * COLUMNS * 4;
  static constexpr int PER_SM = C::THREADS > 512 || SMEM > 113 * 1024 ? 1 : 2;
};
template <typename TI, int T>
__global__ void __launch_bounds__(WideNorm<TI, T>::C::THREADS, 1024 / WideNorm<TI, T>::C::THREADS)
    norm_wide_rows_kernel(const TI *x, int64_t ldx, const void *weight, const void *bias,
                          int param_dtype, void *y, int64_t ldy, int out_dtype, float *mean_out,
                          float *rstd_out, float eps, int64_t M, int64_t N) {
  using K = WideNorm<TI, T>;
  constexpr int G = K::C::GROUPS, PIECE_WORDS = K::WORDS / kWidePieces;
  __shared__ float red[G][2][T / 32];
  extern __shared__ uint4 dyn[];
  const typename K::Ring ring{dyn};
  // weight, bias: [which][piece][half of the piece][t] of four columns
  float4 *params = reinterpret_cast<float4 *>(dyn + K::Ring::BYTES / 16);
  const int g = threadIdx.x / T, t = threadIdx.x % T;
  const float n = static_cast<float>(N), inv_n = 1.0f / n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + g;
  auto columns = [&](int c) { return Columns<T, true>{static_cast<int64_t>(c) * T * VEC, N, t}; };
  auto fetch = [&](int64_t i, int stage) {
    if (i < M) {
#pragma unroll
      for (int c = 0; c < kWidePieces; ++c)
        if (columns(c).in(0)) {
#pragma unroll
          for (int k = 0; k < PIECE_WORDS; ++k)
            ring.copy(stage, c * PIECE_WORDS + k,
                      reinterpret_cast<const uint4 *>(x + i * ldx + columns(c).at(0)) + k);
        }
    }
    ring.commit();
  };
  grid_dependency_wait();
  grid_launch_dependents();
#pragma unroll
  for (int k = 0; k < K::STAGES; ++k) fetch(row + k * step, k);
  if (g == 0) {
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int c = 0; c < kWidePieces; ++c) {
        float p[VEC];
        if (columns(c).in(0)) {
          columns(c).params(which ? bias : weight, param_dtype, which ? 0.0f : 1.0f, p);
          params[((which * kWidePieces + c) * 2) * T + t] = make_float4(p[0], p[1], p[2], p[3]);
          params[((which * kWidePieces + c) * 2 + 1) * T + t] = make_float4(p[4], p[5], p[6], p[7]);
        }
      }
  }
  __syncthreads();
  for (int stage = 0; row < M; row += step) {
    float v[kWidePieces][VEC];
    float s = 0.0f;
    ring.wait();
#pragma unroll
    for (int c = 0; c < kWidePieces; ++c) {
      alignas(16) TI e[VEC];
#pragma unroll
      for (int k = 0; k < PIECE_WORDS; ++k)
        reinterpret_cast<uint4 *>(e)[k] =
            columns(c).in(0) ? *ring.slot(stage, c * PIECE_WORDS + k) : uint4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[c][i] = to_f32(e[i]);
        s += v[c][i];
      }
    }
    fetch(row + K::STAGES * step, stage);  // into the slots just read
    stage = stage + 1 < K::STAGES ? stage + 1 : 0;
    const float mean = mean_of(group_sum<T>(s, red[g][0], g), n, inv_n);
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < kWidePieces; ++c)
      if (columns(c).in(0)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          v[c][i] -= mean;
          q = fmaf(v[c][i], v[c][i], q);
        }
      }
    const float rstd = rsqrtf(mean_of(group_sum<T>(q, red[g][1], g), n, inv_n) + eps);
#pragma unroll
    for (int c = 0; c < kWidePieces; ++c)
      if (columns(c).in(0)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 w = params[(c * 2 + h) * T + t];
          const float4 b = params[((kWidePieces + c) * 2 + h) * T + t];
          float *o = &v[c][4 * h];
          o[0] = fmaf(o[0] * rstd, w.x, b.x);
          o[1] = fmaf(o[1] * rstd, w.y, b.y);
          o[2] = fmaf(o[2] * rstd, w.z, b.z);
          o[3] = fmaf(o[3] * rstd, w.w, b.w);
        }
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

// One pass for rows a CTA's registers hold: a group of T threads a row, 16 columns a thread in
// two pieces, x and dy read once (the next rows on their way in the ring where rows are 16-byte
// aligned), dx written, and the columns' sums of dy xh and dy kept in registers over all of the
// group's rows. The groups of a CTA join theirs at the end; column_finish adds the CTAs.
//
// 16384 x 4096 bf16 on one GB300, with the finish: 82 us, 4.9 TB/s. Sixteen warps an SM
// (118 registers) leave it waiting for its own row-long chain of loads, sums and barrier (0.47
// instructions issued a cycle and scheduler). Measured and not kept, each with the finish: a
// third ring stage (the same), eight columns a thread with the next row in registers (92 us;
// with the ring it spilled at 64 registers, 100 us), and dx a row behind the sums with both
// recomputed from the ring, three CTAs an SM (99 us).
constexpr int kBackPieces = 2;
template <typename TI, int T, bool VECTOR>
struct NormBackward {
  using C = Cta<T, 256>;
  static constexpr int PIECE_WORDS = VEC * static_cast<int>(sizeof(TI)) / 16;
  static constexpr int WORDS = 2 * kBackPieces * PIECE_WORDS;  // x and dy
  static constexpr int STAGES = 2;
  using Ring = RowRing<WORDS, STAGES, C::THREADS>;
  static constexpr int COLUMNS = T * kBackPieces * VEC;
  // weight, or at the end the groups' sums: two fp32 values a column
  static constexpr int SMEM = (VECTOR ? Ring::BYTES : 0) + 2 * COLUMNS * 4;
  static constexpr int PER_SM = 512 / C::THREADS;  // 128 registers a thread
};
template <typename TI, int T, bool VECTOR>
__global__ void __launch_bounds__(Cta<T, 256>::THREADS, 512 / Cta<T, 256>::THREADS)
    norm_backward_kernel(const TI *__restrict__ dy, int64_t lddy, const TI *__restrict__ x,
                         int64_t ldx, const void *weight, int param_dtype,
                         const float *__restrict__ mean, const float *__restrict__ rstd,
                         TI *__restrict__ dx, int64_t lddx, float *__restrict__ partials,
                         int32_t M, int64_t N) {
  using K = NormBackward<TI, T, VECTOR>;
  constexpr int G = K::C::GROUPS, PW = K::PIECE_WORDS;
  __shared__ float red[G][2][2 * (T / 32)];
  extern __shared__ uint4 dyn[];
  const typename K::Ring ring{dyn};
  float4 *ws = reinterpret_cast<float4 *>(dyn + (VECTOR ? K::Ring::BYTES / 16 : 0));
  const int g = threadIdx.x / T, t = threadIdx.x % T;
  const float n = static_cast<float>(N), inv_n = 1.0f / n;
  const int step = static_cast<int>(gridDim.x) * G;
  int row = static_cast<int>(blockIdx.x) * G + g;
  auto columns = [&](int c) { return Columns<T, VECTOR>{static_cast<int64_t>(c) * T * VEC, N, t}; };
  auto after = [&](int i, int k) {  // the group's k-th row from row i on, or M
    const int64_t v = i + static_cast<int64_t>(k) * step;
    return v < M ? static_cast<int>(v) : M;
  };
  auto fetch = [&](int i, int stage) {
    if (i < M) {
#pragma unroll
      for (int c = 0; c < kBackPieces; ++c)
        if (columns(c).in(0)) {
#pragma unroll
          for (int k = 0; k < PW; ++k) {
            ring.copy(stage, 2 * c * PW + k, reinterpret_cast<const uint4 *>(x + i * ldx + columns(c).at(0)) + k);
            ring.copy(stage, (2 * c + 1) * PW + k,
                      reinterpret_cast<const uint4 *>(dy + i * lddy + columns(c).at(0)) + k);
          }
        }
    }
    ring.commit();
  };
  F2 dw[kBackPieces][VEC / 2], db[kBackPieces][VEC / 2];
  float nmu = 0.0f, nr = 0.0f;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row < M) {
    if (VECTOR) {
#pragma unroll
      for (int k = 0; k < K::STAGES; ++k) fetch(after(row, k), k);
    }
    nmu = mean[row], nr = rstd[row];
  }
  if (g == 0) {
#pragma unroll
    for (int c = 0; c < kBackPieces; ++c) {
      float w[VEC];
      columns(c).params(weight, param_dtype, 1.0f, w);
      ws[(2 * c) * T + t] = make_float4(w[0], w[1], w[2], w[3]);
      ws[(2 * c + 1) * T + t] = make_float4(w[4], w[5], w[6], w[7]);
    }
  }
  __syncthreads();
  for (int buf = 0, stage = 0; row < M; buf ^= 1) {
    const F2 mu(-nmu, -nmu), r(nr, nr);
    F2 xh[kBackPieces][VEC / 2], d[kBackPieces][VEC / 2], s0, s1;
    if (VECTOR) ring.wait();
#pragma unroll
    for (int c = 0; c < kBackPieces; ++c) {
      alignas(16) TI ex[VEC];
      alignas(16) TI ed[VEC];
      if (VECTOR) {
#pragma unroll
        for (int k = 0; k < PW; ++k) {
          const bool in = columns(c).in(0);
          reinterpret_cast<uint4 *>(ex)[k] = in ? *ring.slot(stage, 2 * c * PW + k) : uint4{0, 0, 0, 0};
          reinterpret_cast<uint4 *>(ed)[k] = in ? *ring.slot(stage, (2 * c + 1) * PW + k) : uint4{0, 0, 0, 0};
        }
      } else {
        columns(c).load(x + row * ldx, ex);
        columns(c).load(dy + row * lddy, ed);
      }
      const float4 w0 = ws[(2 * c) * T + t], w1 = ws[(2 * c + 1) * T + t];
      const F2 w[VEC / 2] = {F2(w0.x, w0.y), F2(w0.z, w0.w), F2(w1.x, w1.y), F2(w1.z, w1.w)};
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {  // (dy reads as 0 past the row's end)
        xh[c][i] = (F2(to_f32(ex[2 * i]), to_f32(ex[2 * i + 1])) + mu) * r;
        const F2 e(to_f32(ed[2 * i]), to_f32(ed[2 * i + 1]));
        dw[c][i] = fma2(e, xh[c][i], dw[c][i]);
        db[c][i] = db[c][i] + e;
        d[c][i] = e * w[i];
        s0 = s0 + d[c][i];
        s1 = fma2(d[c][i], xh[c][i], s1);
      }
    }
    if (VECTOR) {
      fetch(after(row, K::STAGES), stage);  // into the slots just read
      stage ^= 1;
    }
    const int next = after(row, 1);
    if (next < M) nmu = mean[next], nr = rstd[next];
    const float2 s = group_sum2<T>(s0.get().x + s0.get().y, s1.get().x + s1.get().y, red[g][buf], g);
    if (dx) {
      const float a = -mean_of(s.x, n, inv_n), b = -mean_of(s.y, n, inv_n);
      const F2 a2(a, a), b2(b, b);
#pragma unroll
      for (int c = 0; c < kBackPieces; ++c) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 v = (r * fma2(xh[c][i], b2, d[c][i] + a2)).get();
          o[2 * i] = v.x, o[2 * i + 1] = v.y;
        }
        columns(c).store(dx + row * lddx, o);
      }
    }
    row = next;
  }
  if (!partials) return;
  float sums[2][kBackPieces][VEC];  // of dy xh, of dy
#pragma unroll
  for (int c = 0; c < kBackPieces; ++c)
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 w = dw[c][i].get(), b = db[c][i].get();
      sums[0][c][2 * i] = w.x, sums[0][c][2 * i + 1] = w.y;
      sums[1][c][2 * i] = b.x, sums[1][c][2 * i + 1] = b.y;
    }
  if (G > 1) {  // joined in the groups' order, over the weight's place
    float *join = reinterpret_cast<float *>(ws);
    for (int k = 0; k < G; ++k) {
      __syncthreads();
      if (g == k) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
          for (int c = 0; c < kBackPieces; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              float *at = join + which * K::COLUMNS + (c * VEC + i) * T + t;
              sums[which][c][i] = *at = k ? *at + sums[which][c][i] : sums[which][c][i];
            }
      }
    }
    if (g != G - 1) return;  // the last group holds the sums
  }
  float *out = partials + static_cast<int64_t>(blockIdx.x) * 2 * N;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int c = 0; c < kBackPieces; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (columns(c).in(i)) out[which * N + columns(c).at(i)] = sums[which][c][i];
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
  Columns<32, VECTOR> cols{0, N, static_cast<int>(threadIdx.x % 32)};
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; row < M;
       row += static_cast<int64_t>(gridDim.x) * 8) {
    const float mu = mean[row], r = rstd[row];
    float a = 0.0f, b = 0.0f;
    for (cols.first = 0; cols.first < N; cols.first += 32 * VEC) {
      float vx[VEC], vd[VEC], w[VEC];
      cols.load_f32(x + row * ldx, vx);
      cols.load_f32(dy + row * lddy, vd);
      cols.params(weight, param_dtype, 1.0f, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = vd[i] * w[i];  // 0 past the row's end: dy reads as 0 there
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
  __shared__ float red[2][8][32 * VEC];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const Columns<32, VECTOR> cols{static_cast<int64_t>(blockIdx.x) * 32 * VEC, N, lane};
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * band;
  const int64_t hi = lo + band < M ? lo + band : M;
  float w[VEC], dw[VEC], db[VEC];
  cols.params(weight, param_dtype, 1.0f, w);
#pragma unroll
  for (int i = 0; i < VEC; ++i) dw[i] = db[i] = 0.0f;
  if (cols.in(0)) {
#pragma unroll 2
    for (int64_t row = lo + warp; row < hi; row += 8) {
      float vx[VEC], vd[VEC];
      cols.load_f32(x + row * ldx, vx);
      cols.load_f32(dy + row * lddy, vd);
      const float mu = mean[row], r = rstd[row];
      const float2 m = means[row];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float xh = (vx[i] - mu) * r;
        dw[i] = fmaf(vd[i], xh, dw[i]);
        db[i] += vd[i];
        vx[i] = r * (fmaf(vd[i], w[i], -m.x) - xh * m.y);
      }
      if (dx) cols.store(dx + row * lddx, vx);
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
  if (cols.in(i)) {
    float *out = partials + static_cast<int64_t>(blockIdx.y) * 2 * N + cols.at(i);
    out[0] = a;
    out[N] = b;
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

template <typename TI, int T>
void launch_rows(const NormArgs &a) {
  using C = Cta<T, 256>;
  const int grid = grid_of((a.M + C::GROUPS - 1) / C::GROUPS, a.sm_count, 1024 / C::THREADS);
  auto kernel = a.vec ? norm_rows_kernel<TI, T, true> : norm_rows_kernel<TI, T, false>;
  launch_pdl(kernel, dim3(grid), C::THREADS, 0, a.s, static_cast<const TI *>(a.x), a.ldx, a.weight,
             a.bias, a.param_dtype, a.y, a.ldy, a.out_dtype, a.mean, a.rstd, a.eps, a.M, a.N);
}

template <typename TI, int T>
void launch_wide_rows(const NormArgs &a) {
  using K = WideNorm<TI, T>;
  const int grid = grid_of((a.M + K::C::GROUPS - 1) / K::C::GROUPS, a.sm_count, K::PER_SM);
  auto kernel = norm_wide_rows_kernel<TI, T>;
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM);
  launch_pdl(kernel, dim3(grid), K::C::THREADS, K::SMEM, a.s, static_cast<const TI *>(a.x), a.ldx,
             a.weight, a.bias, a.param_dtype, a.y, a.ldy, a.out_dtype, a.mean, a.rstd, a.eps, a.M, a.N);
}

// Threads that hold a row of N columns, `each` a thread: 32 .. 1024.
int row_threads(int64_t N, int each) {
  int t = 32;
  while (t < 1024 && static_cast<int64_t>(t) * each < N) t *= 2;
  return t;
}

template <typename TI>
void dispatch_rows(const NormArgs &a) {
  // Wide threads from eight rows an SM on: fewer rows leave most of their groups idle and take
  // one row's time, which narrow threads make shorter. Rows past narrow threads' 8192 columns
  // go to wide ones in any number.
  const bool wide = a.vec && a.N > 256 && a.N <= 512 * 32 &&
                    (a.M >= 8 * static_cast<int64_t>(a.sm_count) || a.N > 1024 * VEC);
  if (wide) {
    switch (row_threads(a.N, kWidePieces * VEC)) {
      case 32: return launch_wide_rows<TI, 32>(a);
      case 64: return launch_wide_rows<TI, 64>(a);
      case 128: return launch_wide_rows<TI, 128>(a);
      case 256: return launch_wide_rows<TI, 256>(a);
      default: return launch_wide_rows<TI, 512>(a);
    }
  }
  if (a.N > 1024 * VEC) {
    auto kernel = a.vec ? norm_long_rows_kernel<TI, true> : norm_long_rows_kernel<TI, false>;
    kernel<<<grid_of(a.M, a.sm_count, 64), 512, 0, a.s>>>(
        static_cast<const TI *>(a.x), a.ldx, a.weight, a.bias, a.param_dtype, a.y, a.ldy,
        a.out_dtype, a.mean, a.rstd, a.eps, a.M, a.N);
    return;
  }
  switch (row_threads(a.N, VEC)) {
    case 32: return launch_rows<TI, 32>(a);
    case 64: return launch_rows<TI, 64>(a);
    case 128: return launch_rows<TI, 128>(a);
    case 256: return launch_rows<TI, 256>(a);
    case 512: return launch_rows<TI, 512>(a);
    default: return launch_rows<TI, 1024>(a);
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

template <typename TI, int T, bool VECTOR>
void launch_backward(const NormBackwardArgs &a) {
  using K = NormBackward<TI, T, VECTOR>;
  auto kernel = norm_backward_kernel<TI, T, VECTOR>;
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM);
  launch_pdl(kernel, dim3(a.grid), K::C::THREADS, K::SMEM, a.s, static_cast<const TI *>(a.dy),
             a.lddy, static_cast<const TI *>(a.x), a.ldx, a.weight, a.param_dtype, a.mean, a.rstd,
             static_cast<TI *>(a.dx), a.lddx, a.partials, static_cast<int32_t>(a.M), a.N);
}
template <typename TI, int T>
void launch_backward(const NormBackwardArgs &a) {
  a.vec ? launch_backward<TI, T, true>(a) : launch_backward<TI, T, false>(a);
}

// The one-pass kernel takes rows of up to 512 threads; its grid: as many CTAs as stay on the
// SMs, or as have rows.
constexpr int64_t kOnePassColumns = 512 * kBackPieces * VEC;
int backward_grid(int64_t M, int64_t N, int sm_count) {
  const int t = row_threads(N, kBackPieces * VEC);
  const int64_t groups = t < 256 ? 256 / t : 1;
  return grid_of((M + groups - 1) / groups, sm_count, t < 512 ? 2 : 1);
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
  const bool vec = N % VEC == 0 && aligned16(dy, lddy, esize(grad_dtype)) &&
                   aligned16(x, ldx, is) && aligned16(dx, lddx, is) && aligned16(weight, 0, 4);
  if (N <= kOnePassColumns && grad_dtype == in_dtype) {
    float *sums = static_cast<float *>(workspace);
    const int grid = backward_grid(M, N, sm_count);
    const NormBackwardArgs a{dy, lddy, x, ldx, weight, param_dtype, mean, rstd, dx, lddx,
                             dweight || dbias ? sums : nullptr, M, N,
                             vec, grid, s};
    FF_TYPED(in_dtype, TI, {
      switch (row_threads(N, kBackPieces * VEC)) {
        case 32: launch_backward<TI, 32>(a); break;
        case 64: launch_backward<TI, 64>(a); break;
        case 128: launch_backward<TI, 128>(a); break;
        case 256: launch_backward<TI, 256>(a); break;
        default: launch_backward<TI, 512>(a); break;
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
