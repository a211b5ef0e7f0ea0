// ff_token_kernel.cu -- products of one to eight tokens with an epilogue, and the gated pair,
// for weights stored [features, K]:
//
//   y_n = act(sum_k x_k w_nk + bias_n) + residual_n    or    h_n = act(x . g_n) * (x . u_n)
//
// The bound is reading the weights once, and at a generation step's sizes (a few us of HBM
// time) nearly as much the time before the first byte and after the last. So there is no
// shared-memory ring, tensor core or cluster to set up: every warp streams the weight rows of
// R features straight into registers, R x U 16-byte loads a lane in flight, multiplies
// them with the tokens' elements (from L1) in fp32, and folds the lanes with shuffles. Where
// features alone do not fill the machine, the warps of a CTA share their K and join through
// shared memory in a fixed order.
//
// On one GB300 the tensor-core kernel (ff_few_kernel.cu) has about 5 us outside the stream,
// this one about 3; on 134 MB of weights the two are level, and this one's multiply-adds grow
// with the tokens (plan_token in ff_launch.cu has the measurements and the rule).
#include "activation.cuh"
#include "ff_kernels.h"
#include "ptx.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// E elements of a row from k, as fp32; elements past K read as 0.
template <typename T, bool VECTOR>
struct Lane {
  // elements a lane takes at a time: 16 bytes, or in rows without that alignment as many
  // single elements, 32 apart, so that a warp still reads whole sectors
  static constexpr int E = 16 / sizeof(T);
  static constexpr int STEP = 32 * E;  // elements a warp takes at a time
  alignas(16) T e[E];
  __device__ __forceinline__ void load(const T *row, int64_t k0, int lane, int64_t K) {
    if (VECTOR) {
      *reinterpret_cast<uint4 *>(e) =
          k0 + lane * E < K ? *reinterpret_cast<const uint4 *>(row + k0 + lane * E) : uint4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int64_t k = k0 + i * 32 + lane;
        e[i] = k < K ? row[k] : from_f32<T>(0.0f);
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return to_f32(e[i]); }
};

// MT tokens, R features a warp (gated: R of each projection), U steps of K in flight.
template <typename T, bool GATED, int MT, int R, int U, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    token_kernel(const TokenParams p) {
  constexpr int S = GATED ? 2 : 1;
  __shared__ float red[kWarps][S * R * MT];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kw = p.k_warps, groups = kWarps / kw;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * groups + warp / kw) * R;
  const T *x = static_cast<const T *>(p.X);
  const T *w[S] = {static_cast<const T *>(p.W)};
  int64_t ldw[S] = {p.ldw};
  if (GATED) w[S - 1] = static_cast<const T *>(p.W2), ldw[S - 1] = p.ldw2;
  using L = Lane<T, VECTOR>;
  const int64_t steps = (p.K + L::STEP - 1) / L::STEP;
  // The weights' first lines are asked into L2 while the previous kernel ends. They are read
  // after the wait, from L2, so that weights which that kernel writes are seen as written.
  // (1 x 4096 x 4096 bf16, calls one after another: 9.5 us without, 9.2 with; 8192^2: no change.)
  if (lane % 8 == 0) {
#pragma unroll
    for (int u = 0; u < 2 * U; ++u) {
      const int64_t k = (warp % kw + static_cast<int64_t>(u) * kw) * L::STEP + lane * L::E;
      if (k >= p.K) break;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t n = n0 + r < p.f.N ? n0 + r : p.f.N - 1;
          prefetch_l2(w[s] + n * ldw[s] + k);
        }
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();
  float acc[S][R][MT];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[s][r][m] = 0.0f;
  // Rows past the last feature or token read the last one again; their sums are not stored.
  for (int64_t i0 = warp % kw; i0 < steps; i0 += static_cast<int64_t>(kw) * U) {
    L wv[U][S][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k0 = (i0 + static_cast<int64_t>(u) * kw) * L::STEP;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t n = n0 + r < p.f.N ? n0 + r : p.f.N - 1;
          wv[u][s][r].load(w[s] + n * ldw[s], k0, lane, p.K);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k0 = (i0 + static_cast<int64_t>(u) * kw) * L::STEP;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        L xv;
        xv.load(x + (m < p.f.M ? m : p.f.M - 1) * p.ldx, k0, lane, p.K);
#pragma unroll
        for (int i = 0; i < L::E; ++i) {
          const float xf = xv[i];
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[s][r][m] = fmaf(wv[u][s][r][i], xf, acc[s][r][m]);
        }
      }
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float v = acc[s][r][m];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) red[warp][(s * MT + m) * R + r] = v;
      }
  __syncthreads();
  // One thread an output: the group's warps in order, then the epilogue.
  const int out = threadIdx.x;
  if (out >= groups * R * MT) return;
  // (features of a token run fastest over the threads)
  const int m = out / (groups * R), f = out % (groups * R);
  const int64_t n = static_cast<int64_t>(blockIdx.x) * groups * R + f;
  if (m >= p.f.M || n >= p.f.N) return;
  float sum[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    sum[s] = 0.0f;
    for (int k = 0; k < kw; ++k) sum[s] += red[f / R * kw + k][(s * MT + m) * R + f % R];
  }
  constexpr bool FAST = sizeof(T) == 2;
  float y;
  if (GATED) {
    if (p.f.pre) {
      store_any(p.f.pre, p.f.out_dtype, m * p.f.ld_pre + n, sum[0]);
      store_any(p.f.pre2, p.f.out_dtype, m * p.f.ld_pre2 + n, sum[S - 1]);
    }
    y = activate_one<FAST>(sum[0], p.f.act) * sum[S - 1];
  } else {
    float z = sum[0];
    if (p.f.bias) z += load_any(p.f.bias, p.f.bias_dtype, n);
    if (p.f.pre) store_any(p.f.pre, p.f.out_dtype, m * p.f.ld_pre + n, z);
    y = activate_one<FAST>(z, p.f.act);
    if (p.f.residual) y += load_any(p.f.residual, p.f.out_dtype, m * p.f.ld_residual + n);
  }
  store_any(p.f.C, p.f.out_dtype, m * p.f.ldc + n, y);
}

template <typename T, bool GATED, int MT, int R, int U>
cudaError_t launch_token(bool vector, const TokenParams &p, cudaStream_t s) {
  auto kernel = vector ? token_kernel<T, GATED, MT, R, U, true> : token_kernel<T, GATED, MT, R, U, false>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dependency_wait
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t per_cta = static_cast<int64_t>(kWarps / p.k_warps) * R;
  cfg.gridDim = dim3(static_cast<unsigned>((p.f.N + per_cta - 1) / per_cta), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Features a warp and steps in flight: 8 loads of 16 bytes a lane. More tokens take more
// features a warp: every one of their elements is loaded (from L1) once for all of them.
template <typename T, bool GATED>
cudaError_t dispatch(bool vector, const TokenParams &p, cudaStream_t s) {
  constexpr int S = GATED ? 2 : 1;
  if (p.f.M <= 1) return launch_token<T, GATED, 1, 2 / S, 4>(vector, p, s);
  if (p.f.M <= 2) return launch_token<T, GATED, 2, 2 / S, 4>(vector, p, s);
  if (p.f.M <= 4) return launch_token<T, GATED, 4, 4 / S, 2>(vector, p, s);
  return launch_token<T, GATED, 8, 4 / S, 2>(vector, p, s);
}

}  // namespace

cudaError_t token_launch(bool gated, int dtype, bool vector, const TokenParams &p, cudaStream_t s) {
  if (p.f.M < 1 || p.f.M > kTokenMax || p.k_warps < 1 || kWarps % p.k_warps) return cudaErrorInvalidValue;
  FF_TYPED(dtype, T, {
    return gated ? dispatch<T, true>(vector, p, s) : dispatch<T, false>(vector, p, s);
  })
  return cudaErrorInvalidValue;
}

}  // namespace ff
}  // namespace gemm_gb300
