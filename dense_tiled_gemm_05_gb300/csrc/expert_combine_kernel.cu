// expert_combine_kernel.cu -- rows back from their experts' order, for long aligned rows:
//
//   y[t] = sum_j w[t, j] z[position[t, j]] + residual[t]
//
// by bulk copies: a warp takes 2 KB of a token's k rows and of its residual at a time (1 KB where
// these are many), all of them copied to shared memory while it adds up the piece before. Sums in
// fp32 in the order of j, the residual last, rounded once: the same bits as combine_kernel
// (expert_rows_kernel.cu), which runs where rows or counts do not fit this one. Positions outside
// [0, rows) are passed over.
//
// Bound by the bytes moved. Registers hold what loads have on the way, shared memory five times as
// much: 16384 tokens of 4 x 4 KB and a residual, bf16 on one GB300, 57 us (6.5 TB/s) against 64; 8192 of
// 2 x 8 KB 42 against 54; 16384 of one 8 KB row 43 against 71. Rows below 1.5 KB do not gain (1 KB: 21 us
// against 19.5; 512 bytes: 17 against 9.7), nor do few pieces (512 tokens of 4 x 4 KB: 3.7 against 3.4).
// The parts of a piece that a shorter one does not fill are added up all the same: tests for them cost
// more (4096 tokens of 8 x 14 KB: 84 us against 80).
#include <algorithm>

#include "activation.cuh"
#include "expert_internal.h"
#include "pdl.h"
#include "tc_common.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

constexpr int kWarps = 4;
constexpr int kPiece = 2048;         // bytes of a row at a time, at most
constexpr int kMostRows = 8;         // of a token
constexpr int kLeastRow = 1536;      // bytes of a row
constexpr int kStage = 10 * 1024;    // a warp's pieces of one token, about
constexpr int kFlight = 164 * 1024;  // all stages of an SM (100: 78 us in the first case above; 200: 57)
constexpr int kCtas = 6;             // an SM, at most

struct BulkParams {
  const void *z;
  int64_t ldz;
  const int32_t *position;
  const void *w;
  int32_t w_dtype, k;
  const void *residual;
  int64_t ldr;
  void *y;
  int64_t ldy, tokens, rows, N;
  int32_t pieces, cols;  // a row's, and the columns of each but the last
  int *status;
  uint64_t timeout_ns;
  int32_t stall;  // test hook: no copy is issued
};

// One piece of one token; a warp's pieces are gridDim.x * kWarps apart.
struct Unit {
  int64_t t;
  int q;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

int esize(int dt) { return dt == GEMM_F32 ? 4 : 2; }

template <typename E>
__device__ __forceinline__ void load8(const E *from, float (&v)[VEC]) {
  alignas(16) E e[VEC];
#pragma unroll
  for (int i = 0; i < VEC * static_cast<int>(sizeof(E)) / 16; ++i)
    reinterpret_cast<uint4 *>(e)[i] = reinterpret_cast<const uint4 *>(from)[i];
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
}

template <typename TI, typename TO, int PIECE>
__global__ void __launch_bounds__(32 * kWarps, kCtas) combine_bulk_kernel(const BulkParams p) {
  constexpr int COLS = PIECE / static_cast<int>(sizeof(TI)), PARTS = COLS / (32 * VEC);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][2];
  __shared__ int abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, k = p.k;
  uint64_t *bar = bars[warp];
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  const TI *z = static_cast<const TI *>(p.z);
  const TO *residual = static_cast<const TO *>(p.residual);
  const uint32_t stage_bytes = static_cast<uint32_t>(k * PIECE + (residual ? COLS * sizeof(TO) : 0));
  uint8_t *own = smem + warp * 2 * stage_bytes;
  const Watchdog wd{&abort_flag, p.status, p.timeout_ns};

  const int pieces = p.pieces;
  const int apart = static_cast<int>(gridDim.x) * kWarps, first = static_cast<int>(blockIdx.x) * kWarps + warp;
  const int dt = apart / pieces, dq = apart - dt * pieces;
  const auto after = [&](Unit u) {
    u.t += dt, u.q += dq;
    if (u.q >= pieces) u.q -= pieces, ++u.t;
    return u;
  };
  // lane j: the token's j-th position and weight
  const auto ask = [&](const Unit &u, int32_t &pos, float &f) {
    const bool there = lane < k && u.t < p.tokens;
    pos = there ? p.position[u.t * k + lane] : -1;
    f = !p.w ? 1.0f : there ? load_any(p.w, p.w_dtype, u.t * k + lane) : 0.0f;
  };
  // Copies of a unit's rows, one a lane; lane 31 has no row and takes the residual. The rows that exist.
  const auto issue = [&](const Unit &u, int32_t pos, int s) {
    const bool mine = pos >= 0 && pos < p.rows;
    const uint32_t has = __ballot_sync(0xffffffffu, mine);
    const int64_t c0 = static_cast<int64_t>(u.q) * p.cols;
    const uint32_t cols = static_cast<uint32_t>(min(static_cast<int64_t>(p.cols), p.N - c0));
    const uint32_t bytes = cols * sizeof(TI), bytes_r = residual ? cols * static_cast<uint32_t>(sizeof(TO)) : 0;
    if (lane == 0) mbar_arrive_expect_tx(&bar[s], __popc(has) * bytes + bytes_r);
    __syncwarp();
    const uint32_t to = smem_u32(own + s * stage_bytes);
    if (p.stall) return has;
    if (mine) bulk_load(to + lane * PIECE, z + pos * p.ldz + c0, bytes, &bar[s]);
    if (lane == 31 && residual) bulk_load(to + k * PIECE, residual + u.t * p.ldr + c0, bytes_r, &bar[s]);
    return has;
  };

  Unit now{first / pieces, first % pieces}, next = after(now);
  int32_t pos, next_pos;
  float f, next_f;
  ask(now, pos, f);
  ask(next, next_pos, next_f);
  uint32_t has = now.t < p.tokens ? issue(now, pos, 0) : 0u;
  int s = 0;
  uint32_t phases = 0;
  while (now.t < p.tokens) {
    const bool more = next.t < p.tokens;
    const uint32_t next_has = more ? issue(next, next_pos, s ^ 1) : 0u;
    const Unit far = after(next);
    float far_f;
    ask(far, next_pos, far_f);
    if (!__all_sync(0xffffffffu, mbar_wait(&bar[s], phases >> s & 1, wd))) {
      // the copies of both stages have landed before this CTA's shared memory is another's
      tc::drain_wait(&bar[s], phases >> s & 1, p.timeout_ns);
      if (more) tc::drain_wait(&bar[s ^ 1], phases >> (s ^ 1) & 1, p.timeout_ns);
      break;
    }
    phases ^= 1u << s;
    float sum[PARTS][VEC];
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
      for (int c = 0; c < VEC; ++c) sum[i][c] = 0.0f;
    // (columns past the piece's: whatever the stage holds, never stored)
    const int64_t c0 = static_cast<int64_t>(now.q) * p.cols;
    const int cols = static_cast<int>(min(static_cast<int64_t>(p.cols), p.N - c0));
    const uint8_t *stage = own + s * stage_bytes;
    for (int j = 0; j < k; ++j) {
      const float wj = __shfl_sync(0xffffffffu, f, j);
      if (!(has >> j & 1)) continue;
      const TI *row = reinterpret_cast<const TI *>(stage + j * PIECE) + lane * VEC;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        float v[VEC];
        load8(row + i * 32 * VEC, v);
#pragma unroll
        for (int c = 0; c < VEC; ++c) sum[i][c] = fmaf(wj, v[c], sum[i][c]);
      }
    }
    if (residual) {
      const TO *row = reinterpret_cast<const TO *>(stage + k * PIECE) + lane * VEC;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        float v[VEC];
        load8(row + i * 32 * VEC, v);
#pragma unroll
        for (int c = 0; c < VEC; ++c) sum[i][c] += v[c];
      }
    }
    TO *y = static_cast<TO *>(p.y) + now.t * p.ldy + c0 + lane * VEC;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
      if (i * 32 * VEC + lane * VEC < cols) {
        alignas(16) TO e[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) e[c] = from_f32<TO>(sum[i][c]);
#pragma unroll
        for (int q = 0; q < VEC * static_cast<int>(sizeof(TO)) / 16; ++q)
          reinterpret_cast<uint4 *>(y + i * 32 * VEC)[q] = reinterpret_cast<const uint4 *>(e)[q];
      }
    __syncwarp();  // the stage has been read
    now = next, next = far;
    f = next_f, next_f = far_f;
    has = next_has;
    s ^= 1;
  }
}

// How a call is cut: the room of a piece, and a row's pieces, of one length but for the last, in whole
// 128-byte lines.
struct Cut {
  int piece;  // bytes at most
  int64_t cols, pieces;
  int smem, ctas;  // a CTA's bytes; CTAs an SM
  Cut(int64_t k, int64_t N, int in_dtype, int out_dtype, bool residual) {
    const int in = esize(in_dtype), out = residual ? esize(out_dtype) : 0;
    piece = kPiece;
    if (piece / in * (k * in + out) > kStage) piece /= 2;
    const int64_t room = piece / in, line = 128 / in, least = (N + room - 1) / room;
    cols = ((N + least - 1) / least + line - 1) / line * line;
    pieces = (N + cols - 1) / cols;
    smem = static_cast<int>(2 * kWarps * room * (k * in + out));
    ctas = std::clamp(kFlight / smem, 1, kCtas);
  }
};

}  // namespace

bool expert_combine_bulk_fits(int64_t tokens, int64_t k, int64_t N, int in_dtype, int out_dtype,
                              bool residual, int sm_count) {
  if (k < 1 || k > kMostRows || N * esize(in_dtype) < kLeastRow) return false;
  const Cut cut(k, N, in_dtype, out_dtype, residual);
  return tokens * cut.pieces >= 2 * static_cast<int64_t>(sm_count) * cut.ctas * kWarps;
}

cudaError_t expert_combine_bulk_launch(const void *z, int64_t ldz, int in_dtype, const int32_t *position,
                                       const void *w, int w_dtype, const void *residual, int64_t ldr,
                                       void *y, int64_t ldy, int out_dtype, int64_t tokens, int64_t k,
                                       int64_t rows, int64_t N, int sm_count, int *status,
                                       uint64_t timeout_ns, bool stall, cudaStream_t s) {
  const Cut cut(k, N, in_dtype, out_dtype, residual != nullptr);
  BulkParams p{};
  p.z = z, p.ldz = ldz, p.position = position, p.w = w, p.w_dtype = w_dtype;
  p.k = static_cast<int32_t>(k);
  p.residual = residual, p.ldr = ldr, p.y = y, p.ldy = ldy;
  p.tokens = tokens, p.rows = rows, p.N = N;
  p.pieces = static_cast<int32_t>(cut.pieces), p.cols = static_cast<int32_t>(cut.cols);
  p.status = status, p.timeout_ns = timeout_ns, p.stall = stall;
  cudaError_t e = cudaSuccess;
  FF_TYPED(in_dtype, TI, {
    FF_TYPED(out_dtype, TO, {
      const auto kernel = cut.piece == kPiece ? combine_bulk_kernel<TI, TO, kPiece>
                                              : combine_bulk_kernel<TI, TO, kPiece / 2>;
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFlight);
      if (e == cudaSuccess)
        launch_pdl(kernel, dim3(static_cast<unsigned>(sm_count * cut.ctas)), 32 * kWarps,
                   static_cast<size_t>(cut.smem), s, p);
    })
  })
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace ff
}  // namespace gemm_gb300
