// ff_launch.cu -- host side of the fused products (ff_few_kernel.cu, ff_pair_kernel.cu): which
// kernel and tile a product takes, copies of operands TMA cannot address, tensor maps, launch.
#include <cstring>

#include "ff_launch.h"

using namespace gemm_gb300::api;

namespace gemm_gb300 {
namespace ff {

namespace {

bool tma_legal(const void *p, int64_t ld, int64_t lines, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (lines <= 1 || (ld * es) % 16 == 0);
}

// rows x cols operand with the K extent along columns (X) or rows (W).
void plan_x(FusedOperand *o, int64_t M, int64_t K, Carve *carve) {
  o->transpose = o->layout == GEMM_COL_MAJOR;
  o->staged = o->transpose || !tma_legal(o->ptr, o->ld, M, 2);
  if (!o->staged) return;
  o->staged_ld = round_up(K, 8);
  o->offset = carve->take(M * o->staged_ld, 2);
}
void plan_w(FusedOperand *o, int64_t K, int64_t N, Carve *carve) {
  const int64_t lines = o->layout == GEMM_ROW_MAJOR ? K : N, len = o->layout == GEMM_ROW_MAJOR ? N : K;
  o->staged = !tma_legal(o->ptr, o->ld, lines, 2);
  if (!o->staged) return;
  o->staged_ld = round_up(len, 8);
  o->offset = carve->take(lines * o->staged_ld, 2);
}

// Tiles and cluster split of the few-token kernel: the token tile, the number of CTAs that
// share a tile's K, and one or two CTAs an SM, with the least estimated time. The estimate, in
// SM cycles: a 64-long K-block of a CTA's tile costs the larger of its MMAs (half a cycle a
// token and K-step, or what their operands take from shared memory) and its bytes at 41 a
// cycle (one SM's TMA stream; two CTAs on an SM get 1.6 times that); the weights and tokens
// together take HBM's rate, and all copies the L2's; and each round of CTAs has its start, its
// epilogue and, for a split tile, the joining of partials. The constants are fitted to 750
// measured configurations of 31 products (one GB300, 1 to 8192 tokens, plain and gated, from
// graphs); over those the choice takes 2.8 % more than the best on average, 27 % at most.
void plan_few(FusedProduct *q, int64_t k_blocks, int sm_count) {
  const int accs = q->gated ? 2 : 1;
  const int64_t sms = sm_count > 0 ? sm_count : 1;
  const int64_t tiles_f = (q->N + kFewFeatures - 1) / kFewFeatures;
  double best = 1e300;
  int64_t narrower = 0;
  for (const int64_t t : {16, 32, 48, 64, 96, 128, 192, 256}) {
    if (narrower >= q->M || (q->gated && t > 128)) break;  // a narrower tile holds all tokens
    narrower = t;
    const int64_t tiles_t = (q->M + t - 1) / t, tiles = tiles_t * tiles_f;
    const double bytes = static_cast<double>(few_stage_bytes(q->gated, static_cast<int>(t)));
    const double mma = 4.4 * accs * (t / 2.0 > 32 + t / 4.0 ? t / 2.0 : 32 + t / 4.0);
    const double kb = mma > bytes / 41 ? mma : bytes / 41;
    const double hbm = static_cast<double>(accs * tiles_f * kFewFeatures + tiles_t * t) * k_blocks * 128 / 3200;
    const double l2 = static_cast<double>(tiles) * k_blocks * bytes / 9000;
    for (int c = 1; c <= 8; c *= 2) {
      if (c > 1 && k_blocks < 2 * c) break;
      const int64_t per_cta = (k_blocks + c - 1) / c;
      for (int per_sm = 1; per_sm <= 2; ++per_sm) {
        const size_t room = static_cast<size_t>(per_sm == 2 ? 112 : 226) * 1024;
        if (few_smem_bytes(q->gated, static_cast<int>(t), 2, c > 1) > room) continue;
        const int64_t one = few_max_clusters(c);
        // (two clusters' CTAs on an SM pack less than twice as many; of four, hardly more)
        const int64_t clusters = per_sm == 1 ? one : c == 1 ? 2 * one : c == 4 ? one * 7 / 5 : one * 9 / 5;
        const int64_t rounds = (tiles + clusters - 1) / clusters;
        // CTAs of the busiest SM in the full rounds and in the last one
        const int64_t full = tiles / clusters, rest = tiles % clusters;
        const int64_t last = (rest * c + sms - 1) / sms < per_sm ? (rest * c + sms - 1) / sms : per_sm;
        auto shared = [](int64_t n) { return n < 2 ? static_cast<double>(n) : n / 1.6; };
        double time = kb * per_cta * (full * shared(per_sm) + shared(last));
        if (time < hbm) time = hbm;
        if (time < l2) time = l2;
        const double tail = c == 1 ? 1100 + 18.0 * accs * t
                                   : 550 + 36.0 * accs * t + 48.0 * accs * t / c + 460.0 * c;
        const double cost = time + rounds * (7700 + tail);
        if (cost < best) {
          best = cost;
          FewParams &p = q->few_params;
          p.tile_t = static_cast<int>(t);
          p.tiles_t = static_cast<int>(tiles_t);
          p.tiles_f = static_cast<int>(tiles_f);
          p.splits = c;
          int64_t stages = static_cast<int64_t>((room - kFewFixedBytes) / few_stage_bytes(q->gated, p.tile_t));
          if (stages > per_cta) stages = per_cta;
          if (stages > 16) stages = 16;
          p.stages = static_cast<int>(stages);
        }
      }
    }
  }
  q->few_cost = best;
}

// The CTA-pair kernel's estimate, in the same cycles: 512 a K-block and round of tiles, and
// about 16000 for the first loads and the last tile's epilogue; a tile's epilogue runs under
// the next one's K-loop unless that is shorter (8000); and no less than HBM's time.
double pair_cost(const FusedProduct &q, int64_t k_blocks, int64_t clusters, int stream_k) {
  const int64_t tiles = q.tiles_m * q.tiles_n;
  double rounds = static_cast<double>((tiles + clusters - 1) / clusters);
  if (tiles > clusters && use_split_k(stream_k, tiles, k_blocks, clusters))
    rounds = static_cast<double>(tiles) / clusters;
  const double loop = 512.0 * k_blocks;
  const double time = loop + (rounds - 1) * (loop > 8000 ? loop : 8000);
  const double hbm = static_cast<double>((q.gated ? 2 : 1) * q.N + q.M) * k_blocks * 128 / 3200;
  return 16000 + (time > hbm ? time : hbm);
}

// The token kernel's rule: weights stored [features, K], one product, and few enough tokens
// that its multiply-adds hide under the stream of weights. Measured on one GB300, us, token
// kernel against few-token kernel: bf16 1 x 1024 x 1024 2.9 / 5.9, 1 x 4096 x 4096 (34 MB of
// weights) 9.3 / 11.3, 1 x 8192 x 8192 (134 MB) 25.7 / 25.0, two tokens 34 MB 9.9 / 11.3, 134
// MB 30 / 24, four tokens 17 MB 6.2 / 8.0, 34 MB 12.2 / 10.8: up to 80 MB of weights times
// tokens. Rows TMA cannot address it reads as they are, where the few-token kernel copies all
// weights first (1 x 4097 x 1001: 4.4 / 22). fp32: up to eight tokens, against the exact
// product on the tensor cores with its 30 us of fixed cost (8 x 4096 x 4096: 45 / 109).
bool plan_token(FusedProduct *q, int sm_count) {
  const int es = esize_of(q->in_dtype);
  if (q->M > kTokenMax || q->K2 > 0 || q->W.layout != GEMM_COL_MAJOR ||
      q->X.layout != GEMM_ROW_MAJOR || q->N > (int64_t{1} << 30))
    return false;
  q->vector = q->K % (16 / es) == 0 && tma_legal(q->X.ptr, q->X.ld, q->M, es) &&
              tma_legal(q->W.ptr, q->W.ld, q->N, es) &&
              (!q->gated || tma_legal(q->W2.ptr, q->W2.ld, q->N, es));
  const int64_t rows = q->gated ? 2 * q->N : q->N;
  if (q->in_dtype != GEMM_F32 &&
      (q->M > 4 || (q->vector && rows * q->K * es * q->M > int64_t{80} << 20)))
    return false;
  // Warps that share a weight row's K, in steps of 512 bytes: eight steps a warp, or down to
  // four where the rows would not make up 24 warps an SM (best of 1, 2, 4, 8 within 10 % on
  // most of the sizes above).
  const int64_t steps = (q->K * es + 511) / 512;
  const int64_t tasks = (rows + (q->M <= 2 ? 1 : 3)) / (q->M <= 2 ? 2 : 4);
  q->k_warps = 1;
  while (q->k_warps < 8 &&
         (steps >= 16 * q->k_warps ||
          (steps >= 8 * q->k_warps && tasks * q->k_warps < 24 * static_cast<int64_t>(sm_count))))
    q->k_warps *= 2;
  q->kind = FusedProduct::kToken;
  return true;
}

// Whether the outputs and the residual allow accesses of four elements.
bool four_wide(const FusedProduct &q) {
  const int es = esize_of(q.out_dtype);
  auto ok = [&](const void *p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && ld % 4 == 0);
  };
  return ok(q.C, q.ldc) && ok(q.ep.pre, q.ep.ld_pre) && ok(q.pre2, q.ld_pre2) &&
         ok(q.ep.residual, q.ep.ld_residual);
}

// Tile and cluster split of the fp32 tile kernel by estimated time in SM cycles -- about 11000
// outside the K-loop, and 45 to 105 multiply-adds a cycle by how many warps an SM holds -- and
// whether that is less than the exact product's on the tensor cores: 32 us, 18 us per 1024 of
// K (the chunk drains; shared out over idle clusters from some 3000 on), the writing and reading
// of the split operands, and 14 us where rows of the output are unaligned. Measured on one GB300, us, this kernel against that (with
// silu and a residual): 512^3 14 / 41, 512 x 1024 x 1024 35 / 51, 1023 x 1025 x 1000 60 / 69,
// 300 x 64 x 4096 26 / 83, 64 x 2048 x 8192 73 / 136, 3000 x 64 x 8192 131 / 146, 2048 x 1024 x 1024 109 / 57, gated
// 1000 x 500 x 1000 61 / 101. It errs where the two are close (1023 x 1000 x 1025 65 / 58) and
// on the longest K (2432 x 64 x 65536 915 / 677).
bool plan_tile(FusedProduct *q, int sm_count) {
  if (!q->exact || q->K2 > 0) return false;
  const int64_t sms = sm_count > 0 ? sm_count : 1;
  const int64_t steps = (q->K + kTileK - 1) / kTileK;
  const int products = q->gated ? 2 : 1;
  double best = 1e300;
  for (const int size : {64, 128}) {
    const int64_t bm = tile_rows(size), bn = tile_cols(q->gated, size);
    const int64_t tiles = ((q->M + bm - 1) / bm) * ((q->N + bn - 1) / bn);
    if (tiles > (int64_t{1} << 26)) continue;
    for (int c = 1; c <= 8; c *= 2) {
      if (c > 1 && steps < 4 * c) break;
      const int64_t busy = (tiles * c + sms - 1) / sms;  // CTAs of the busiest SM
      const double rate = size == 128 ? (busy > 1 ? 105 : 77) : busy > 2 ? 75 : busy > 1 ? 62 : 45;
      // (an SM with more CTAs than the average has the last of them to itself)
      const double ctas = busy > 1 ? 0.5 * (busy + static_cast<double>(tiles * c) / sms) : 1.0;
      const double work = ctas * bm * bn * products * ((steps + c - 1) / c) * kTileK;
      const double join = c > 1 ? (size == 128 ? 7000 : 1500) + 300.0 * c : 0.0;
      const double cost = 11000 + work / rate + join;
      if (cost < best) best = cost, q->tile_size = size, q->tile_splits = c;
    }
  }
  const int64_t tensor_tiles = ((q->M + 255) / 256) * ((q->N + 255) / 256);
  const int64_t clusters = sms > 1 ? sms / 2 : 1;
  const double k1024 = q->K / 1024.0;
  const double loop = (18 * k1024 < 55 ? 18 * k1024 : 55) * ((tensor_tiles + clusters - 1) / clusters);
  const double split = 16.0 * (q->M + q->N) * q->K / 5e6;
  const double ragged = four_wide(*q) && q->N % 4 == 0 ? 0 : 14;  // stores that TMA cannot make
  if (best >= products * 1900.0 * (32 + loop + split + ragged)) return false;
  q->kind = FusedProduct::kTile;
  return true;
}

cudaError_t stage(const FusedOperand &o, int64_t lines, int64_t len, char *buf, cudaStream_t s) {
  if (o.transpose) return transpose_launch(o.ptr, o.ld, buf + o.offset, o.staged_ld, lines, len, 2, s);
  return repack_launch(o.ptr, o.ld, buf + o.offset, o.staged_ld, lines, len, 2, s);
}

}  // namespace

bool plan_fused(gemm_handle_t h, FusedProduct *q, Carve *carve) {
  if (q->M < 1 || q->N < 1 || q->K < 1) return false;
  if (h->force_path == 2) return false;  // the FMA kernel was asked for
  if (q->gated && q->out_dtype != q->in_dtype) return false;
  // (the multiply-add kernels only where no tensor-core kernel is asked for)
  const bool multiply_adds = !h->cta_pair && h->force_path != 1;
  if (multiply_adds && plan_token(q, h->sm_count)) return true;
  if (q->in_dtype == GEMM_F32) return multiply_adds && plan_tile(q, h->sm_count);
  const int64_t k_blocks = (q->K + 63) / 64 + (q->K2 + 63) / 64;
  const int64_t tile_n = q->gated ? 128 : 256;
  q->tiles_m = (q->M + 255) / 256;
  q->tiles_n = (q->N + tile_n - 1) / tile_n;
  const int64_t clusters = pair_slots(h->sm_count, h->max_ctas);
  if (q->tiles_m * q->tiles_n > INT32_MAX / 8 || k_blocks > INT32_MAX) return false;
  // Where the 256-row tiles are few, or few of their rows are tokens, the few-token kernel's
  // smaller tiles, which share their K-loops over clusters, take less time.
  plan_few(q, k_blocks, h->sm_count);
  bool few = q->few_cost < pair_cost(*q, k_blocks, clusters, h->stream_k);
  if (h->cta_pair) few = h->cta_pair == 1;  // GEMM_OPT_CTA_PAIR
  q->kind = few ? FusedProduct::kFew : FusedProduct::kPair;
  plan_x(&q->X, q->M, q->K, carve);
  plan_w(&q->W, q->K, q->N, carve);
  if (q->gated) {
    plan_w(&q->W2, q->K, q->N, carve);
  } else if (q->K2 > 0) {
    plan_x(&q->X2, q->M, q->K2, carve);
    plan_w(&q->W2, q->K2, q->N, carve);
  }
  return true;
}

gemm_status_t run_fused(gemm_handle_t h, const FusedProduct &q, char *buf, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  FusedParams f{};
  f.M = static_cast<int32_t>(q.M), f.N = static_cast<int32_t>(q.N);
  f.out_dtype = q.out_dtype;
  f.act = q.ep.act;
  f.bias = q.ep.bias, f.bias_dtype = q.ep.bias_dtype;
  f.residual = q.ep.residual, f.ld_residual = q.ep.ld_residual;
  f.C = q.C, f.ldc = q.ldc;
  f.pre = q.ep.pre, f.ld_pre = q.ep.ld_pre;
  f.pre2 = q.pre2, f.ld_pre2 = q.ld_pre2;
  f.status = h->status;
  f.timeout_ns = h->timeout_us * 1000ull;
  f.debug_flags = stall_flags(h->stall_producer);
  if (q.kind == FusedProduct::kToken) {
    TokenParams p{};
    p.f = f;
    p.X = q.X.ptr, p.ldx = q.X.ld;
    p.W = q.W.ptr, p.ldw = q.W.ld;
    p.W2 = q.W2.ptr, p.ldw2 = q.W2.ld;
    p.K = q.K;
    p.k_warps = q.k_warps;
    e = token_launch(q.gated, q.in_dtype, q.vector, p, s);
    if (e != cudaSuccess) return cuda_fail(e, "token kernel launch");
    h->launches += 1;
    return GEMM_OK;
  }
  if (q.kind == FusedProduct::kTile) {
    TileParams p{};
    p.f = f;
    p.X = static_cast<const float *>(q.X.ptr), p.ldx = q.X.ld, p.x_k = q.X.layout == GEMM_ROW_MAJOR;
    p.W = static_cast<const float *>(q.W.ptr), p.ldw = q.W.ld, p.w_k = q.W.layout == GEMM_COL_MAJOR;
    p.W2 = static_cast<const float *>(q.W2.ptr), p.ldw2 = q.W2.ld;
    p.K = q.K;
    p.splits = q.tile_splits;
    p.run_steps = tile_run_steps(q.K);
    p.vec = four_wide(q);
    e = tile_launch(q.gated, q.tile_size, p, s);
    if (e != cudaSuccess) return cuda_fail(e, "fp32 tile kernel launch");
    h->launches += 1;
    return GEMM_OK;
  }
  const bool few = q.kind == FusedProduct::kFew;
  const bool two_x = !q.gated && q.K2 > 0, two_w = q.gated || q.K2 > 0;
  struct Use {
    const FusedOperand *o;
    bool used, w;
    int64_t K;
  };
  const Use uses[4] = {{&q.X, true, false, q.K}, {&q.W, true, true, q.K}, {&q.X2, two_x, false, q.K2},
                       {&q.W2, two_w, true, q.gated ? q.K : q.K2}};
  // Operand boxes are one 128-byte row of K (or, for row-major weights, of N) wide.
  const uint32_t x_rows = few ? static_cast<uint32_t>(q.few_params.tile_t) : 128u;
  CUtensorMap maps[4];
  for (int i = 0; i < 4; ++i) {
    if (!uses[i].used) {
      maps[i] = maps[i & 1];  // never read
      continue;
    }
    const FusedOperand &o = *uses[i].o;
    const bool w = uses[i].w, row = o.layout == GEMM_ROW_MAJOR;
    // as stored: `lines` lines of `len` contiguous elements
    int64_t lines = w ? (row ? uses[i].K : q.N) : (row ? q.M : uses[i].K);
    int64_t len = w ? (row ? q.N : uses[i].K) : (row ? uses[i].K : q.M);
    const void *ptr = o.ptr;
    int64_t ld = o.ld;
    if (o.staged) {
      e = stage(o, lines, len, buf, s);
      if (e != cudaSuccess) return cuda_fail(e, "stage operand");
      h->launches += 1;
      ptr = buf + o.offset;
      ld = o.staged_ld;
      if (o.transpose) {
        const int64_t t = lines;
        lines = len, len = t;
      }
    }
    const uint32_t rows = w ? (row ? 64u : 128u) : x_rows;
    if (!encode_2d(&maps[i], q.in_dtype, ptr, len, lines, ld, 64, rows)) return GEMM_ERR_CUDA;
  }
  f.kb_first = static_cast<int32_t>((q.K + 63) / 64);
  f.k_blocks = f.kb_first + static_cast<int32_t>(two_x ? (q.K2 + 63) / 64 : 0);
  const bool w_mn = q.W.layout == GEMM_ROW_MAJOR;
  const int os = esize_of(q.out_dtype);
  if (few) {
    FewParams p = q.few_params;
    p.f = f;
    p.f.idesc = make_idesc(q.in_dtype, w_mn, false, p.tile_t, 128);
    p.vec = four_wide(q);
    e = few_launch(q.gated, w_mn, maps[0], maps[1], maps[2], maps[3], p, s);
    if (e != cudaSuccess) return cuda_fail(e, "few-token kernel launch");
    h->launches += 1;
    return GEMM_OK;
  }
  PairMaps pm;
  std::memset(&pm, 0, sizeof pm);
  pm.X = maps[0], pm.W = maps[1], pm.X2 = maps[2], pm.W2 = maps[3];
  PairParams p{};
  p.f = f;
  p.f.idesc = make_idesc(q.in_dtype, false, w_mn, 256, 256);
  p.tiles_m = static_cast<int32_t>(q.tiles_m), p.tiles_n = static_cast<int32_t>(q.tiles_n);
  p.group_m = h->group_m < p.tiles_m ? h->group_m : p.tiles_m;
  // TMA stores only where rows end on 16-byte boundaries (see the planner)
  p.tma_out = (q.N * os) % 16 == 0;
  const void *outs[4] = {q.C, f.pre, f.pre2, f.residual};
  const int64_t lds[4] = {q.ldc, f.ld_pre, f.ld_pre2, f.ld_residual};
  CUtensorMap *out_maps[4] = {&pm.C, &pm.Z, &pm.Z2, &pm.R};
  for (int i = 0; i < 4; ++i)
    p.tma_out = p.tma_out && (!outs[i] || tma_legal(outs[i], lds[i], 2, os));
  for (int i = 0; i < 4 && p.tma_out; ++i)
    if (outs[i] && !encode_2d(out_maps[i], q.out_dtype, outs[i], q.N, q.M, lds[i],
                              static_cast<uint32_t>(128 / os), 32))
      return GEMM_ERR_CUDA;
  const int64_t fit = tc2_max_active_clusters();
  if (fit <= 0) return GEMM_ERR_CUDA;
  const int64_t tiles = q.tiles_m * q.tiles_n;
  int64_t slots = pair_slots(h->sm_count, h->max_ctas);
  if (slots > fit) slots = fit;
  const int32_t t32 = static_cast<int32_t>(tiles), s32 = static_cast<int32_t>(slots);
  p.sk_dp_tiles = sk_dp_tiles(t32, p.f.k_blocks, s32, use_split_k(h->stream_k, tiles, p.f.k_blocks, slots));
  if (p.sk_dp_tiles < t32) {
    const gemm_status_t st = split_workspace(h, slots, 256, &p.sk_epoch_word, &p.sk_flags,
                                             &p.sk_partials, &pm.P, s);
    if (st != GEMM_OK) return st;
  } else if (slots > tiles) {
    slots = tiles;
  }
  e = pair_launch(q.gated, w_mn, pm, p, static_cast<int>(2 * slots), s);
  if (e != cudaSuccess) return cuda_fail(e, "fused product launch");
  h->launches += 1;
  return GEMM_OK;
}

}  // namespace ff
}  // namespace gemm_gb300
