// expert_launch.cu -- host side of the experts' products (expert_pair_kernel.cu,
// expert_grad_kernel.cu, expert_f32_kernel.cu): copies of operands TMA cannot address, tensor maps, launch.
#include <cstring>

#include "expert_launch.h"

using namespace gemm_gb300::api;

namespace gemm_gb300 {
namespace ff {

namespace {

constexpr int ES = 2;  // bytes an element of the tensor cores' operands
// Rows an expert, on average, up to which products run in narrow tiles. The host knows no counts: all
// experts are taken to have rows. Where they do, the weights' stream is the time; where a few of many
// have them all, narrow tiles cost (256 experts, 4096 x 2048, one GB300, us: 8192 rows, narrow, over all
// experts, eight and one: 640, 123 and 124; 8193 rows, wide: 651, 85 and 84).
constexpr int64_t kNarrowRows = 32;

bool addressable(const void *p, int64_t lines, int64_t ld, int64_t count, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (lines <= 1 || (ld * ES) % 16 == 0) &&
         (count <= 1 || (stride * ES) % 16 == 0);
}

// Boxes are one 128-byte row of K (or, with the features inside, of N) wide.
bool encode_rows(CUtensorMap (&m)[4], const ExpertOperand &x, int dtype) {
  for (uint32_t i = 0; i < 4; ++i)
    if (!encode_2d(&m[i], dtype, x.ptr, x.len, x.lines, x.ld, 64, 32 * (i + 1))) return false;
  return true;
}
bool encode_weights(CUtensorMap *m, const ExpertOperand &w, bool mn, bool panels, int dtype) {
  if (panels) return encode_4d_panels(m, dtype, w.ptr, w.len, w.lines, w.ld, w.count, w.stride, 64, 2);
  return encode_3d(m, dtype, w.ptr, w.len, w.lines, w.count, w.ld, w.stride, 64, mn ? 64 : 128);
}
// Rows as an operand whose sum runs over them.
bool encode_outer(CUtensorMap *m, const ExpertOperand &x, int dtype, int32_t *panels) {
  *panels = x.len % 64 == 0 && x.lines > 1;
  return *panels ? encode_3d_panels(m, dtype, x.ptr, x.len, x.lines, x.ld, 64, 2, false)
                 : encode_2d(m, dtype, x.ptr, x.len, x.lines, x.ld, 64, 64);
}

// The handle's workspace of split tiles: [epoch word, arrival count | eight flags a CTA of the largest
// grid | sums of `clusters`]. The region of the flags has one size for all grids, so that none finds
// sums where it expects flags.
gemm_status_t share_workspace(gemm_handle_t h, ExpertParams *p, int64_t clusters, bool narrow, cudaStream_t s) {
  const int64_t ctas = 2 * static_cast<int64_t>(h->sm_count);
  const size_t flags = static_cast<size_t>(round_up(static_cast<int64_t>((2 + 8 * ctas) * sizeof(int)), 256));
  const size_t sums = static_cast<size_t>(clusters * expert_share_floats(narrow)) * sizeof(float);
  const gemm_status_t st = reserve(h, h->expert_split, flags + sums, s, flags);
  if (st != GEMM_OK) return st;
  p->sk_epoch_word = static_cast<int *>(h->expert_split.ptr);
  p->sk_flags = p->sk_epoch_word + 2;
  p->sk_partials = reinterpret_cast<float *>(static_cast<char *>(h->expert_split.ptr) + flags);
  return GEMM_OK;
}

// Narrow tiles run two CTAs an SM. (The occupancy query counts one; were a cluster to wait for its
// place, those that run do not wait for it: sums come from lower-numbered clusters.)
int64_t clusters_of(gemm_handle_t h, int64_t tiles, bool narrow) {
  int64_t n = pair_slots(h->sm_count, h->max_ctas);
  const int64_t fit = expert_max_clusters();
  if (n > fit) n = fit;
  if (narrow && h->max_ctas == 0) n *= 2;
  return n > tiles ? tiles : n;
}

}  // namespace

void ExpertOperand::plan(Carve *carve) {
  staged = lines > 0 && len > 0 && !addressable(ptr, lines, ld, count, stride);
  if (staged) offset = carve->take(count * lines * round_up(len, 8), ES);
}

gemm_status_t ExpertOperand::stage(gemm_handle_t h, char *buf, cudaStream_t s, const int32_t *offsets) {
  if (!staged) return GEMM_OK;
  const int64_t to_ld = round_up(len, 8);
  char *to = buf + offset;
  const cudaError_t err = expert_stage_launch(ptr, ld, stride, lines, count, len, to, to_ld, offsets, s);
  if (err != cudaSuccess) return cuda_fail(err, "stage operand");
  h->launches += 1;
  ptr = to, ld = to_ld, stride = lines * to_ld;
  staged = false;
  return GEMM_OK;
}

ExpertOperand expert_weights(const void *W, int64_t ld, int64_t stride, int64_t experts, int64_t K,
                             int64_t N, int layout) {
  ExpertOperand o;
  o.ptr = W, o.ld = ld, o.count = experts, o.stride = stride;
  o.lines = layout == GEMM_ROW_MAJOR ? K : N;
  o.len = layout == GEMM_ROW_MAJOR ? N : K;
  return o;
}

ExpertOperand expert_rows(const void *X, int64_t ld, int64_t rows, int64_t cols) {
  ExpertOperand o;
  o.ptr = X, o.ld = ld, o.lines = rows, o.len = cols;
  return o;
}

bool expert_tiles_fit(int64_t experts, int64_t rows, int64_t N, int64_t K) {
  const int64_t n = (N + 63) / 64, k = (K + 63) / 64, t = rows / 64 + experts;
  const int64_t most = INT32_MAX / 4;
  return t <= most / n && t <= most / k && n <= most / k && experts <= most / (n * k);
}

gemm_status_t run_expert(gemm_handle_t h, const ExpertProduct &q, cudaStream_t s) {
  ExpertMaps maps;
  std::memset(&maps, 0, sizeof maps);
  const bool two_x = q.second, two_w = q.second || q.gated;
  const bool panels = q.w_mn && q.N % 64 == 0 && q.W.lines > 1;
  // The interleaved pair's map leads from one matrix to the other: less than 2^40 bytes, the limit
  // of a tensor map's strides, and the same steps in both.
  const intptr_t apart = reinterpret_cast<intptr_t>(q.W2.ptr) - reinterpret_cast<intptr_t>(q.W.ptr);
  const ExpertMode mode = !q.gated ? kExpertPlain
                          : !q.w_mn && q.N % 16 == 0 && q.W.ld == q.W2.ld &&
                                  (q.experts == 1 || q.W.stride == q.W2.stride) && apart != 0 &&
                                  apart > -(intptr_t{1} << 40) && apart < (intptr_t{1} << 40)
                              ? kExpertMixed
                              : kExpertTwo;
  bool ok = encode_rows(maps.X, q.X, q.dtype) && (!two_x || encode_rows(maps.X2, q.X2, q.dtype));
  if (ok && mode == kExpertMixed)
    ok = encode_mixed(&maps.W, q.dtype, apart > 0 ? q.W.ptr : q.W2.ptr, apart > 0 ? apart : -apart, q.W.len,
                      q.W.lines, q.W.count, q.W.ld, q.W.stride, 64, 4);
  else if (ok)
    ok = encode_weights(&maps.W, q.W, q.w_mn, panels, q.dtype) &&
         (!two_w || encode_weights(&maps.W2, q.W2, q.w_mn, panels, q.dtype));
  if (!ok) return GEMM_ERR_CUDA;
  if (!two_x) std::memcpy(maps.X2, maps.X, sizeof maps.X);  // never read
  if (!two_w || mode == kExpertMixed) maps.W2 = maps.W;
  ExpertParams p{};
  p.offsets = q.offsets;
  p.experts = static_cast<int32_t>(q.experts), p.rows = static_cast<int32_t>(q.rows);
  p.N = static_cast<int32_t>(q.N);
  p.kb_first = static_cast<int32_t>((q.K + 63) / 64);
  p.k_blocks = p.kb_first * (q.second ? 2 : 1);
  p.idesc = make_idesc(q.dtype, q.w_mn, false, 0, 256);
  p.dtype = q.dtype, p.act = q.act, p.panels = panels, p.up_first = apart < 0;
  p.C = q.C, p.ldc = q.ldc;
  p.pre = q.pre, p.ld_pre = q.ld_pre, p.pre2 = q.pre2, p.ld_pre2 = q.ld_pre2;
  const auto eights = [](const void *rows, int64_t ld) {
    return reinterpret_cast<uintptr_t>(rows) % 8 == 0 && (ld * ES) % 8 == 0;
  };
  p.wide = q.N % 4 == 0 && eights(q.C, q.ldc) &&
           (!q.pre || (eights(q.pre, q.ld_pre) && eights(q.pre2, q.ld_pre2)));
  p.status = h->status;
  p.timeout_ns = h->timeout_us * 1000ull;
  p.debug_flags = stall_flags(h->stall_producer);
  // at most one part tile an expert, and no more experts with rows than rows
  const int64_t used = q.experts < q.rows ? q.experts : q.rows;
  const bool narrow = mode != kExpertTwo && q.rows <= kNarrowRows * used;
  const int64_t tiles = (q.rows / expert_tokens(mode, narrow) + used) *
                        ((q.N + expert_features(mode) - 1) / expert_features(mode));
  // as many clusters as run at once: how many tiles there are, and whether they are shared, shows
  // on the device
  const int64_t clusters = clusters_of(h, tiles * ((p.k_blocks + 3) / 4), narrow);
  p.stream_k = h->stream_k;
  const gemm_status_t st = share_workspace(h, &p, clusters, narrow, s);
  if (st != GEMM_OK) return st;
  const cudaError_t e = expert_launch(mode, q.w_mn, narrow, maps, p, static_cast<int>(2 * clusters), s);
  if (e != cudaSuccess) return cuda_fail(e, "expert product launch");
  h->launches += 1;
  return GEMM_OK;
}

gemm_status_t run_expert_grad(gemm_handle_t h, const ExpertGrad &q, cudaStream_t s) {
  ExpertGradMaps maps;
  std::memset(&maps, 0, sizeof maps);
  ExpertGradParams p{};
  p.offsets = q.offsets;
  p.experts = static_cast<int32_t>(q.experts), p.rows = static_cast<int32_t>(q.rows);
  p.MA = static_cast<int32_t>(q.A.len), p.NB = static_cast<int32_t>(q.B.len);
  p.tiles_m = (p.MA + 255) / 256, p.tiles_n = (p.NB + 255) / 256;
  p.idesc = make_idesc(q.dtype, true, true, 256, 256);
  p.dtype = q.dtype;
  p.D = q.D, p.ldd = q.ldd, p.stride_d = q.stride_d;
  p.status = h->status;
  p.timeout_ns = h->timeout_us * 1000ull;
  p.debug_flags = stall_flags(h->stall_producer);
  // TMA stores only where lines end on 16-byte boundaries (see the planner)
  p.tma_out = (q.B.len * ES) % 16 == 0 && addressable(q.D, q.A.len, q.ldd, q.experts, q.stride_d);
  if (!encode_outer(&maps.A, q.A, q.dtype, &p.panels_a) || !encode_outer(&maps.B, q.B, q.dtype, &p.panels_b) ||
      (p.tma_out && !encode_3d(&maps.D, q.dtype, q.D, q.B.len, q.A.len, q.experts, q.ldd, q.stride_d, 64, 32)))
    return GEMM_ERR_CUDA;
  const int64_t tiles = q.experts * p.tiles_m * p.tiles_n;
  const cudaError_t e = expert_grad_launch(maps, p, static_cast<int>(2 * clusters_of(h, tiles, false)), s);
  if (e != cudaSuccess) return cuda_fail(e, "expert gradient launch");
  h->launches += 1;
  return GEMM_OK;
}

gemm_status_t run_expert_f32(gemm_handle_t h, const ExpertProduct &q, bool add, cudaStream_t s) {
  ExpertF32Params p{};
  p.offsets = q.offsets;
  p.experts = static_cast<int32_t>(q.experts), p.rows = static_cast<int32_t>(q.rows);
  p.N = static_cast<int32_t>(q.N), p.K = q.K;
  p.A = static_cast<const float *>(q.X.ptr), p.a_line = q.X.ld, p.a_step = 1;
  p.B = static_cast<const float *>(q.W.ptr), p.stride_b = q.W.stride;
  p.b_line = q.w_mn ? 1 : q.W.ld, p.b_step = q.w_mn ? q.W.ld : 1;
  p.C = static_cast<float *>(q.C), p.ldc = q.ldc;
  p.add = add;
  const cudaError_t e = expert_f32_launch(false, p, h->sm_count, s);
  if (e != cudaSuccess) return cuda_fail(e, "expert fp32 product launch");
  h->launches += 1;
  return GEMM_OK;
}

gemm_status_t run_expert_grad_f32(gemm_handle_t h, const ExpertGrad &q, cudaStream_t s) {
  ExpertF32Params p{};
  p.offsets = q.offsets;
  p.experts = static_cast<int32_t>(q.experts), p.rows = static_cast<int32_t>(q.rows);
  p.M = static_cast<int32_t>(q.A.len), p.N = static_cast<int32_t>(q.B.len);
  p.A = static_cast<const float *>(q.A.ptr), p.a_line = 1, p.a_step = q.A.ld;
  p.B = static_cast<const float *>(q.B.ptr), p.b_line = 1, p.b_step = q.B.ld;
  p.C = static_cast<float *>(q.D), p.ldc = q.ldd, p.stride_c = q.stride_d;
  const cudaError_t e = expert_f32_launch(true, p, h->sm_count, s);
  if (e != cudaSuccess) return cuda_fail(e, "expert fp32 gradient launch");
  h->launches += 1;
  return GEMM_OK;
}

}  // namespace ff
}  // namespace gemm_gb300
