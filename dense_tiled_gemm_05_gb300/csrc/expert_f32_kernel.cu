// expert_f32_kernel.cu -- the experts' products in fp32, on fused multiply-adds:
//
//   C[r] (+)= A[r] B[e]            for the rows r of each expert e        (rows)
//   C[e]   = sum_r A[r]^T B[r]     over its rows                          (gradients of weights)
//
// 64 x 64 tiles, 128 threads of 8 x 4 sums in packed multiply-adds, 16 of the summed axis a step; the
// next step's operands are on their way in registers while this one's are multiplied. One stride of
// each operand is 1; alignment is any. A thread's sums move to a running total every 128 steps of the
// axis, so that no addend takes more than 128 + K / 128 roundings. Bound by the instructions around
// the multiply-adds, at 0.6 of the rate that a library's fp32 product reaches on these units (one
// GB300, 16 experts of 1024 rows, 4096 x 2048: 6.6 ms, 42 TFLOP/s; four experts of one row, 1024 x
// 1024: 50 us). Three CTAs an SM: two take 7.4 ms there and four 6.2, but 157 and 219 us against 205
// with 8 experts of 64 rows, 2048 x 2048. 256 threads of 4 x 4 sums, unpacked: 8.1 ms.
#include <algorithm>

#include "activation.cuh"
#include "expert_kernels.h"
#include "expert_tiles.cuh"
#include "pdl.h"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int T = 64;     // rows and columns of a tile
constexpr int STEP = 16;  // of the summed axis
constexpr int kThreads = 128;
constexpr int RUN = 128 / STEP;

// A step of an operand in registers, its elements spread over the threads, and its way to shared
// memory as [STEP][T]. ALONG: the summed axis is the contiguous one (step 1), else the tile's own.
// (T + 4 is a multiple of four, so that lines of shared memory start on 16-byte boundaries.)
template <bool ALONG>
struct Piece {
  static constexpr int PER = T * STEP / kThreads;
  static constexpr int OWN = ALONG ? kThreads / STEP : 0, SUM = ALONG ? 0 : kThreads / T;  // apart
  const float *next;  // this thread's first element of the next step
  int64_t apart, ahead;
  int own, sum, lines;
  float v[PER];

  // From element (0, k0) of the tile's `lines` lines; i is `line` and k `step` elements apart.
  __device__ __forceinline__ Piece(const float *base, int64_t line, int64_t step, int64_t k0, int lines)
      : own(static_cast<int>(threadIdx.x) / (ALONG ? STEP : 1) % T),
        sum(ALONG ? static_cast<int>(threadIdx.x) % STEP : static_cast<int>(threadIdx.x) / T),
        lines(lines) {
    next = base + own * line + (k0 + sum) * step;
    apart = ALONG ? OWN * line : SUM * step;
    ahead = STEP * step;
  }
  // The next STEP of the summed axis, of which `left` are there; other elements are 0.
  __device__ __forceinline__ void load(int64_t left) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = own + OWN * i < lines && sum + SUM * i < left ? next[i * apart] : 0.0f;
    next += ahead;
  }
  __device__ __forceinline__ void store(float (*to)[T + 4]) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) to[sum + SUM * i][own + OWN * i] = v[i];
  }
};

template <bool GRAD, bool ALONG_A, bool ALONG_B>
__global__ void __launch_bounds__(kThreads, 3) expert_f32_kernel(const ExpertF32Params p) {
  __shared__ int32_t tables[2 * (kMaxExperts + 1)];
  __shared__ __align__(16) float a[2][STEP][T + 4];  // read four at a time
  __shared__ __align__(16) float b[2][STEP][T + 4];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tiles_m = (p.M + T - 1) / T, tiles_n = (p.N + T - 1) / T;
  const ExpertTiles table{tables, tables + kMaxExperts + 1, p.experts, tiles_n, T};
  int tiles = p.experts * tiles_m * tiles_n;
  if (!GRAD) {
    table.fill(p.offsets, p.rows, kThreads);
    __syncthreads();
    tiles = table.count();
  }
  // a warp: 32 columns, eight lanes of four, by four lines of four and those 32 further on
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int x0 = 32 * (warp % 2) + 4 * (lane % 8), y0 = 16 * (warp / 2) + 4 * (lane / 8);
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const float *from_a = p.A, *from_b = p.B;
    float *c = p.C;
    int64_t begin = 0, end = p.K;
    int lines, n0;
    if (GRAD) {
      const int per = tiles_m * tiles_n, e = t / per, i = t - e * per;
      const int m0 = i % tiles_m * T;
      n0 = i / tiles_m * T;
      begin = max(0, min(p.offsets[e], p.rows));
      end = max(static_cast<int64_t>(min(p.offsets[e + 1], p.rows)), begin);
      lines = min(T, p.M - m0);
      from_a += m0 * p.a_line;
      from_b += n0 * p.b_line;
      c += e * p.stride_c + m0 * p.ldc + n0;
    } else {
      const ExpertTiles::Tile tile = table.at(t);
      n0 = tile.column * T;
      lines = tile.rows;
      from_a += tile.row0 * p.a_line;
      from_b += tile.e * p.stride_b + n0 * p.b_line;
      c += tile.row0 * p.ldc + n0;
    }
    const int cols = min(T, p.N - n0);
    Piece<ALONG_A> pa(from_a, p.a_line, p.a_step, begin, lines);
    Piece<ALONG_B> pb(from_b, p.b_line, p.b_step, begin, cols);
    F2 total[4][4], run[4][4];  // [pair of lines][column]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) total[i][j] = run[i][j] = both(0.0f);
    pa.load(end - begin);
    pb.load(end - begin);
    int steps = 0;
    __syncthreads();  // the previous tile has been read
    for (int64_t k0 = begin; k0 < end; k0 += STEP) {
      const int stage = ++steps % 2;  // (read two steps ago: the barrier between was passed since)
      pa.store(a[stage]);
      pb.store(b[stage]);
      __syncthreads();
      if (k0 + STEP < end) {
        pa.load(end - k0 - STEP);
        pb.load(end - k0 - STEP);
      }
#pragma unroll
      for (int k = 0; k < STEP; ++k) {
        alignas(16) float x[4];
        alignas(16) F2 y[4];
        *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(&b[stage][k][x0]);
        *reinterpret_cast<ulonglong2 *>(y) = *reinterpret_cast<const ulonglong2 *>(&a[stage][k][y0]);
        *reinterpret_cast<ulonglong2 *>(y + 2) = *reinterpret_cast<const ulonglong2 *>(&a[stage][k][y0 + 32]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 xj = both(x[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) run[i][j] = fma2(y[i], xj, run[i][j]);
        }
      }
      if (steps % RUN == 0 || k0 + STEP >= end) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[i][j] = total[i][j] + run[i][j], run[i][j] = both(0.0f);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = y0 + i / 4 * 32 + i % 4, n = x0 + j;
        if (m < lines && n < cols) {
          float *to = c + m * p.ldc + n;
          const float2 pair = total[i / 2][j].get();
          const float v = i % 2 ? pair.y : pair.x;
          *to = p.add ? *to + v : v;
        }
      }
  }
}

}  // namespace

cudaError_t expert_f32_launch(bool grad, const ExpertF32Params &p, int sm_count, cudaStream_t s) {
  const int64_t lines = grad ? static_cast<int64_t>(p.experts) * ((p.M + T - 1) / T)
                             : p.rows / T + std::min(p.experts, p.rows);  // of tiles, at most
  const int64_t tiles = lines * ((p.N + T - 1) / T), most = static_cast<int64_t>(sm_count) * 16;
  const dim3 grid(static_cast<unsigned>(std::min(tiles, most)));
  const auto kernel = grad            ? expert_f32_kernel<true, false, false>
                      : p.b_step == 1 ? expert_f32_kernel<false, true, true>
                                      : expert_f32_kernel<false, true, false>;
  launch_pdl(kernel, grid, kThreads, 0, s, p);
  return cudaGetLastError();
}

}  // namespace ff
}  // namespace gemm_gb300
