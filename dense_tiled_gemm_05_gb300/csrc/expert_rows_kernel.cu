// expert_rows_kernel.cu -- rows to their experts' order and back:
//
//   y[position[t, j]] = x[t]                                          (gather)
//   y[t]  = sum_j w[t, j] z[position[t, j]] + residual[t]             (combine; see also
//                                                                 expert_combine_kernel.cu)
//   dz[position[t, j]] = w[t, j] dy[t],  dw[t, j] = dy[t] . z[position[t, j]]
//
// and the copies of operands that TMA cannot address.
//
// All are bound by the bytes they move. A warp covers 256 columns, eight a lane, in 16-byte
// accesses where the rows allow it. It reads a token's positions (and weights) with one load,
// lane j the j-th, and hands them round by shuffles, so that all of a token's rows are on the
// way at once. Each row is read and written once; every output element belongs to one lane,
// which adds in the order of j in fp32 and rounds once. Positions outside [0, rows) are passed
// over: nothing is read or written for them. Pairs with one position write its row both, each
// element at some time.
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
constexpr int kCols = 32 * VEC;  // columns a warp covers at a time
constexpr int kWalkers = 4;      // CTAs an SM of kernels whose warps walk tokens
// CTAs of one of many matrices that are copied, at most. One that is passed over costs their starts:
// products of 2001 x 4096 with 32 experts, us, one row of four of them and two rows of each: 53 and 295;
// with 152 CTAs 62 and 303, with 608 50 and 295, but 54 against 34 for one row of 8 of 64, 1001 x 1408.
constexpr int64_t kStageCtas = 304;

bool aligned16(const void *p, int64_t ld, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0);
}
int esize(int dt) { return dt == GEMM_F32 ? 4 : 2; }

// Column blocks along x, tokens along y. Where rows are mostly written, one token a warp: CTAs then
// start in the order of memory, which HBM writes faster than grids that stay and stride through it
// (65536 rows of 4 KB from 16384: 54 us against 63 with 608 CTAs that loop).
dim3 token_grid(int64_t tokens, int64_t N) {
  const int64_t gx = (N + kCols - 1) / kCols, gy = (tokens + kWarps - 1) / kWarps;
  return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>(gy, 65535)));
}
// Where they are mostly read, exactly as many CTAs as stay (16384 tokens of 4 x 4 KB and a residual
// through this file's kernel: 64 us; with two and a half times as many 72), whose warps walk tokens.
dim3 walk_grid(int64_t tokens, int64_t N, int sm_count) {
  const int64_t all = static_cast<int64_t>(sm_count > 0 ? sm_count : 1) * kWalkers;
  const int64_t gx = (N + kCols - 1) / kCols, gy = (tokens + kWarps - 1) / kWarps;
  return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(std::max<int64_t>(std::min(gy, all / gx), 1)));
}

#define FF_TOKENS(t, tokens)                                                              \
  for (int64_t t = static_cast<int64_t>(blockIdx.y) * kWarps + threadIdx.x / 32; t < tokens; \
       t += static_cast<int64_t>(gridDim.y) * kWarps)

// Row of a position, or -1.
__device__ __forceinline__ int64_t row_of(int32_t position, int64_t rows) {
  return position >= 0 && position < rows ? position : -1;
}

template <typename E, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    gather_kernel(const E *__restrict__ x, int64_t ldx, const int32_t *__restrict__ position,
                  E *__restrict__ y, int64_t ldy, int64_t tokens, int k, int64_t rows, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x % 32;
  const RowPiece<VECTOR> cols(static_cast<int64_t>(blockIdx.x) * kCols, N, lane);
  FF_TOKENS(t, tokens) {
    alignas(16) E e[VEC];
    cols.load(x + t * ldx, e);
    for (int j0 = 0; j0 < k; j0 += 32) {
      const int n = min(32, k - j0);
      const int32_t p = lane < n ? position[t * k + j0 + lane] : -1;
      for (int j = 0; j < n; ++j) {
        const int64_t r = row_of(__shfl_sync(0xffffffffu, p, j), rows);
        if (r >= 0) cols.store_raw(y + r * ldy, e);
      }
    }
  }
}

template <typename TI, typename TO, bool VECTOR>
__global__ void __launch_bounds__(kThreads, kWalkers)
    combine_kernel(const TI *__restrict__ z, int64_t ldz, const int32_t *__restrict__ position,
                   const void *__restrict__ w, int w_dtype, const TO *residual, int64_t ldr, TO *y,
                   int64_t ldy, int64_t tokens, int k, int64_t rows, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x % 32;
  const RowPiece<VECTOR> cols(static_cast<int64_t>(blockIdx.x) * kCols, N, lane);
  constexpr int BATCH = sizeof(TI) == 4 || !VECTOR ? 2 : 4;  // rows on the way at once
  const int64_t step = static_cast<int64_t>(gridDim.y) * kWarps;
  int64_t t = static_cast<int64_t>(blockIdx.y) * kWarps + threadIdx.x / 32;
  // a token's first 32 positions and weights are asked for while the token before it is added up
  auto position_of = [&](int64_t i, int j) { return j < k && i < tokens ? position[i * k + j] : -1; };
  auto weight_of = [&](int64_t i, int j) {
    return !w ? 1.0f : j < k && i < tokens ? load_any(w, w_dtype, i * k + j) : 0.0f;
  };
  int32_t next_p = position_of(t, lane);
  float next_f = weight_of(t, lane);
  for (; t < tokens; t += step) {
    float sum[VEC];
    alignas(16) TO res[VEC];  // (y may be the residual: a lane reads its columns before it writes them)
    if (residual) cols.load(residual + t * ldr, res);
#pragma unroll
    for (int c = 0; c < VEC; ++c) sum[c] = 0.0f;
    int32_t p = next_p;
    float f = next_f;
    next_p = position_of(t + step, lane);
    next_f = weight_of(t + step, lane);
    for (int j0 = 0; j0 < k; j0 += 32) {
      const int n = min(32, k - j0);
      if (j0 > 0) p = position_of(t, j0 + lane), f = weight_of(t, j0 + lane);
      for (int j = 0; j < n; j += BATCH) {
        alignas(16) TI e[BATCH][VEC];
        float wj[BATCH];
        bool has[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const int from = min(j + b, 31);
          const int64_t r = row_of(__shfl_sync(0xffffffffu, p, from), rows);
          wj[b] = __shfl_sync(0xffffffffu, f, from);
          has[b] = j + b < n && r >= 0;
          if (has[b]) cols.load(z + r * ldz, e[b]);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
          if (has[b]) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) sum[c] = fmaf(wj[b], to_f32(e[b][c]), sum[c]);
          }
      }
    }
    if (residual) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) sum[c] += to_f32(res[c]);
    }
    cols.store(y + t * ldy, sum);
  }
}

// `share` warps (1, 2, 4 or 8) take the row of one pair (t, j) together, 256 columns each in
// turn, and add their sums in their order. The pairs of a token are neighbours, so that its dy
// comes from L1 after the first.
template <typename TG, typename TZ, bool VECTOR>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const TG *__restrict__ dy, int64_t lddy, const TZ *__restrict__ z,
                            int64_t ldz, const int32_t *__restrict__ position,
                            const void *__restrict__ w, int w_dtype, TZ *__restrict__ dz,
                            int64_t lddz, void *__restrict__ dw, int64_t tokens, int k, int64_t rows,
                            int64_t N, int share) {
  __shared__ float part[kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per_cta = kWarps / share, slot = warp / share, part_of = warp % share;
  const int64_t pairs = tokens * k;
  // (the CTA's warps walk together: barriers below)
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * per_cta; i0 < pairs;
       i0 += static_cast<int64_t>(gridDim.x) * per_cta) {
    const int64_t i = i0 + slot;
    float dot = 0.0f;
    if (i < pairs) {
      const int64_t t = i / k;
      const int64_t r = row_of(position[i], rows);
      if (r >= 0) {
        const float f = w ? load_any(w, w_dtype, i) : 1.0f;
#pragma unroll 2
        for (int64_t c0 = static_cast<int64_t>(part_of) * kCols; c0 < N;
             c0 += static_cast<int64_t>(share) * kCols) {
          const Columns<32, VECTOR> cols{c0, N, lane};
          float g[VEC], v[VEC];
          cols.load_f32(dy + t * lddy, g);
          if (dw) {
            cols.load_f32(z + r * ldz, v);
#pragma unroll
            for (int c = 0; c < VEC; ++c) dot = fmaf(g[c], v[c], dot);
          }
          if (dz) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[c] = f * g[c];
            cols.store(dz + r * lddz, v);
          }
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int d = 16; d; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (share == 1) {
      if (lane == 0 && i < pairs) store_any(dw, w_dtype, i, dot);
      continue;
    }
    if (lane == 0) part[warp] = dot;
    __syncthreads();
    if (part_of == 0 && lane == 0 && i < pairs) {
      for (int q = 1; q < share; ++q) dot += part[warp + q];
      store_any(dw, w_dtype, i, dot);
    }
    __syncthreads();
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads)
    zero_kernel(E *__restrict__ y, int64_t ldy, const int32_t *__restrict__ offsets, int experts,
                int64_t rows, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t lo = max(offsets[0], 0), hi = min(static_cast<int64_t>(offsets[experts]), rows);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (col >= N) return;
  for (int64_t r = lo + blockIdx.y; r < hi; r += gridDim.y) y[r * ldy + col] = from_f32<E>(0.0f);
}

// h = act(g) * u of the experts' rows in fp32; h may be g.
__global__ void __launch_bounds__(kThreads)
    gated_rows_kernel(const float *g, int64_t ldg, const float *__restrict__ u, int64_t ldu, float *h,
                      int64_t ldh, int act, const int32_t *__restrict__ offsets, int experts, int64_t rows,
                      int64_t F) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t lo = max(offsets[0], 0), hi = min(static_cast<int64_t>(offsets[experts]), rows);
  const RowPiece<false> cols(static_cast<int64_t>(blockIdx.x) * kCols, F, threadIdx.x % 32);
  for (int64_t r = lo + static_cast<int64_t>(blockIdx.y) * kWarps + threadIdx.x / 32; r < hi;
       r += static_cast<int64_t>(gridDim.y) * kWarps) {
    float a[VEC], b[VEC];
    cols.load_f32(g + r * ldg, a);
    cols.load_f32(u + r * ldu, b);
    activate_all<false>(a, act);
#pragma unroll
    for (int c = 0; c < VEC; ++c) a[c] *= b[c];
    cols.store(h + r * ldh, a);
  }
}

// A warp copies 256 elements of a line, a lane eight: their 4-byte words, shifted by half a word
// where the line starts on an odd element, as one 16-byte store. At a line's ends its own half of a
// word is read. (32 matrices of 2048 x 1001, a quarter of a gigabyte read and written: about 60 us;
// with two-byte accesses 230.) With offsets, matrices of experts without rows are passed over.
__global__ void __launch_bounds__(kThreads)
    stage_kernel(const uint16_t *__restrict__ src, int64_t ld, int64_t stride, int64_t lines, int64_t len,
                 int64_t chunks, uint16_t *__restrict__ dst, int64_t to_ld,
                 const int32_t *__restrict__ offsets) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t e = blockIdx.y;
  if (offsets && offsets[e + 1] <= offsets[e]) return;
  src += e * stride;
  dst += e * lines * to_ld;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; i < lines * chunks;
       i += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t line = i / chunks;
    const int64_t j0 = (i - line * chunks) * kCols + lane * VEC;
    if (j0 >= len) continue;
    const uint16_t *from = src + line * ld + j0;
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(from) / 2 % 2);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(from - odd);
    const uint16_t *halves = from - odd;
    uint32_t w[5];
#pragma unroll
    for (int q = 0; q < 5; ++q) {
      const int64_t j = j0 - odd + 2 * q;  // the word's first element
      w[q] = 0u;
      if (q == 4 && !odd) break;
      if (j >= 0 && j + 1 < len)
        w[q] = words[q];
      else if (j < 0)
        w[q] = static_cast<uint32_t>(halves[2 * q + 1]) << 16;
      else if (j < len)
        w[q] = halves[2 * q];
    }
    uint4 out;
    out.x = odd ? __funnelshift_r(w[0], w[1], 16) : w[0];
    out.y = odd ? __funnelshift_r(w[1], w[2], 16) : w[1];
    out.z = odd ? __funnelshift_r(w[2], w[3], 16) : w[2];
    out.w = odd ? __funnelshift_r(w[3], w[4], 16) : w[3];
    *reinterpret_cast<uint4 *>(dst + line * to_ld + j0) = out;
  }
}

}  // namespace

cudaError_t expert_stage_launch(const void *src, int64_t ld, int64_t stride, int64_t lines, int64_t count,
                                int64_t len, void *dst, int64_t to_ld, const int32_t *offsets, cudaStream_t s) {
  const int64_t chunks = (len + kCols - 1) / kCols;
  const int64_t ctas =
      std::min<int64_t>((lines * chunks + kWarps - 1) / kWarps, count == 1 ? 1 << 20 : kStageCtas);
  launch_pdl(stage_kernel, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(count)), kThreads, 0, s,
             static_cast<const uint16_t *>(src), ld, stride, lines, len, chunks, static_cast<uint16_t *>(dst),
             to_ld, offsets);
  return cudaGetLastError();
}

cudaError_t expert_gated_rows_launch(const float *g, int64_t ldg, const float *u, int64_t ldu, float *h,
                                     int64_t ldh, int act, const int32_t *offsets, int64_t experts,
                                     int64_t rows, int64_t F, cudaStream_t s) {
  launch_pdl(gated_rows_kernel, token_grid(rows, F), kThreads, 0, s, g, ldg, u, ldu, h, ldh, act, offsets,
             static_cast<int>(experts), rows, F);
  return cudaGetLastError();
}

cudaError_t expert_zero_launch(void *y, int64_t ldy, int es, const int32_t *offsets, int64_t experts,
                               int64_t rows, int64_t N, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((N + kThreads - 1) / kThreads),
                  static_cast<unsigned>(std::min<int64_t>(rows, 1024)));
  if (es == 4)
    launch_pdl(zero_kernel<float>, grid, kThreads, 0, s, static_cast<float *>(y), ldy, offsets,
               static_cast<int>(experts), rows, N);
  else
    launch_pdl(zero_kernel<__half>, grid, kThreads, 0, s, static_cast<__half *>(y), ldy, offsets,
               static_cast<int>(experts), rows, N);
  return cudaGetLastError();
}

cudaError_t expert_gather_launch(const void *x, int64_t ldx, const int32_t *position, void *y,
                                 int64_t ldy, int es, int64_t tokens, int64_t k, int64_t rows,
                                 int64_t N, cudaStream_t s) {
  const bool vector = aligned16(x, ldx, es) && aligned16(y, ldy, es) && N % VEC == 0;
  auto go = [&](auto *type, auto vec) {
    using E = std::remove_pointer_t<decltype(type)>;
    launch_pdl(gather_kernel<E, decltype(vec)::value>, token_grid(tokens, N), kThreads, 0, s,
               static_cast<const E *>(x), ldx, position, static_cast<E *>(y), ldy, tokens,
               static_cast<int>(k), rows, N);
  };
  if (es == 4)
    vector ? go(static_cast<float *>(nullptr), std::true_type{}) : go(static_cast<float *>(nullptr), std::false_type{});
  else
    vector ? go(static_cast<__half *>(nullptr), std::true_type{}) : go(static_cast<__half *>(nullptr), std::false_type{});
  return cudaGetLastError();
}

cudaError_t expert_combine_launch(const void *z, int64_t ldz, int in_dtype, const int32_t *position,
                                  const void *w, int w_dtype, const void *residual, int64_t ldr,
                                  void *y, int64_t ldy, int out_dtype, int64_t tokens, int64_t k,
                                  int64_t rows, int64_t N, int sm_count, int *status, uint64_t timeout_ns,
                                  bool stall, cudaStream_t s) {
  const bool vector = aligned16(z, ldz, esize(in_dtype)) && aligned16(y, ldy, esize(out_dtype)) &&
                      aligned16(residual, ldr, esize(out_dtype)) && N % VEC == 0;
  if (vector && expert_combine_bulk_fits(tokens, k, N, in_dtype, out_dtype, residual != nullptr, sm_count))
    return expert_combine_bulk_launch(z, ldz, in_dtype, position, w, w_dtype, residual, ldr, y, ldy, out_dtype,
                                      tokens, k, rows, N, sm_count, status, timeout_ns, stall, s);
  FF_TYPED(in_dtype, TI, {
    FF_TYPED(out_dtype, TO, {
      auto go = [&](auto kernel) {
        launch_pdl(kernel, walk_grid(tokens, N, sm_count), kThreads, 0, s, static_cast<const TI *>(z), ldz,
                   position, w, w_dtype, static_cast<const TO *>(residual), ldr,
                   static_cast<TO *>(y), ldy, tokens, static_cast<int>(k), rows, N);
      };
      vector ? go(combine_kernel<TI, TO, true>) : go(combine_kernel<TI, TO, false>);
    })
  })
  return cudaGetLastError();
}

cudaError_t expert_combine_backward_launch(const void *dy, int64_t lddy, int grad_dtype,
                                           const void *z, int64_t ldz, const int32_t *position,
                                           const void *w, int w_dtype, void *dz, int64_t lddz,
                                           int in_dtype, void *dw, int64_t tokens, int64_t k,
                                           int64_t rows, int64_t N, int sm_count, cudaStream_t s) {
  const int is = esize(in_dtype);
  const bool vector = aligned16(dy, lddy, esize(grad_dtype)) && aligned16(dw ? z : nullptr, ldz, is) &&
                      aligned16(dz, lddz, is) && N % VEC == 0;
  // A pair's row is shared by warps while they have columns and the pairs alone do not fill the GPU.
  const int64_t pairs = tokens * k, target = static_cast<int64_t>(sm_count > 0 ? sm_count : 1) * 32;
  int share = 1;
  while (share < kWarps && pairs * share < target && N > static_cast<int64_t>(share) * kCols) share *= 2;
  const int per_cta = kWarps / share;
  const int64_t ctas = std::min<int64_t>((pairs + per_cta - 1) / per_cta, int64_t{1} << 20);
  FF_TYPED(grad_dtype, TG, {
    FF_TYPED(in_dtype, TZ, {
      auto go = [&](auto kernel) {
        launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), kThreads, 0, s,
                   static_cast<const TG *>(dy), lddy, static_cast<const TZ *>(z), ldz, position, w,
                   w_dtype, static_cast<TZ *>(dz), lddz, dw, tokens, static_cast<int>(k), rows, N, share);
      };
      vector ? go(combine_backward_kernel<TG, TZ, true>) : go(combine_backward_kernel<TG, TZ, false>);
    })
  })
  return cudaGetLastError();
}

}  // namespace ff
}  // namespace gemm_gb300
