// expert_pair_kernel.cu -- the experts' products of rows sorted by expert:
//
//   Y[r] = X[r] W[e] (+ X2[r] W2[e])      or      H[r] = act(X[r] Wg[e]) * (X[r] Wu[e])
//
// for the rows r in [offsets[e], offsets[e + 1]) of each expert e.
//
// How many rows an expert has is known on the device only, from none to all of them, so tiles
// have to fit any count. The weights are the MMA's M side, 256 output features on a pair of CTAs
// (tcgen05.mma.cta_group::2), and the tokens its N side, whose width is set for every tile: an
// expert's rows are shared evenly over tiles of at most 256, each a multiple of 32 wide. 256-row
// tiles of tokens would waste half a tile an expert on average, an eighth of the time at 1024 rows
// and a third at 256. The same layout serves few tokens: a 32-column MMA, and the time is that of
// the weights' stream.
//
// Grid: one cluster of two CTAs for every two SMs, which walk the tiles of all experts; every CTA
// makes the table of tiles in its shared memory from the offsets, so that no count goes to the host
// and no other launch is needed. Token tiles run fastest: the clusters at work share weights
// through L2, and the next tile's loads and MMAs run under a tile's epilogue (two accumulators).
// Where the last round of tiles would leave clusters idle for long, or there are fewer tiles than
// clusters, the last tiles' K-blocks are shared equally (sk_schedule.h): a cluster that lacks a
// tile's end writes its fp32 sums, one 128-byte line a column and warp, and the cluster that has
// the end adds them in their order.
//
// The gated pair of K-contiguous weights: one TMA copy brings 16 rows of the gate's weights, the
// same 16 of the up projection's, the next 16 of the gate's and so on (a 5D map whose third axis
// leads from one matrix to the other), so that a warp's 32 TMEM lanes are g and u of 16 features
// and a shuffle brings them together: 128 features a tile, one MMA a K-step. Other weights (other
// layouts, feature counts that are no multiple of 16) run as two MMAs a K-step against the same
// 128 tokens, g and u in the same lanes of two column ranges: those narrower MMAs read a third more
// shared memory an operation (16 experts of 1024 rows, 2048 x 4096: 1840 TFLOP/s, interleaved 1940;
// with g and u kept 1695 and 1825).
//
// Measured on one GB300, short runs: 16384 rows, 4096 x 2048, one expert 1900 to 1945 TFLOP/s, 16 of
// 1024 rows 1800 to 1830, 16 of 46 to 4407 rows 1690 (back to back, at the power cap: 1650, 1550 and
// 1450); 256 rows of 32 experts, 4096 x 2048: 80 us for 540 MB.
//
// The epilogue has one feature a lane and tokens along its registers, which lanes exchange for wider
// stores (store_tokens). Rows past the expert's last are not stored (they are the next expert's).
// Bound: tensor cores for many rows an expert, HBM for few, the epilogue for K below some 1000.
#include <atomic>

#include "activation.cuh"
#include "expert_kernels.h"
#include "expert_tiles.cuh"

namespace gemm_gb300 {
namespace ff {
namespace {

using namespace tc;

constexpr int BM = 128;                         // features per CTA
constexpr int BK = 64;
constexpr int W_BYTES = BM * kRowBytes;         // one weight box (MN-major: two panels)
constexpr int PANEL_BYTES = BK * kRowBytes;
constexpr int kEpi = 8;                         // epilogue warps
constexpr int kExpertThreads = 64 + 32 * kEpi;
// A kernel's tiles and shared memory. Narrow: for few rows an expert, tiles of at most 64 tokens, so
// that two CTAs fit an SM: twice as many, smaller shares of the weights' stream, and a kernel's start
// (the table, the first loads) runs under the end of the one before it. One GB300, us, calls one
// after another, narrow and wide: 4 rows gated 2048 x 4096 26.9 and 29.7, 256 rows of 32
// experts 4096 x 2048 81.8 and 86.0.
template <int MODE, bool NARROW>
struct Shape {
  static constexpr bool TWO = MODE == kExpertTwo;             // weight boxes, accumulators
  static constexpr int FEATURES = expert_features(MODE) / 2;  // a CTA's
  static constexpr int TOKENS = expert_tokens(MODE, NARROW);
  static constexpr int ACC = NARROW ? 64 : 256;               // TMEM columns of a tile (two: half each)
  static constexpr int W_ALL = (TWO ? 2 : 1) * W_BYTES;
  static constexpr int STAGE = W_ALL + TOKENS / 2 * kRowBytes;  // (a CTA's half of the tokens)
  static constexpr int STAGES = TWO || NARROW ? 5 : 6;
  static constexpr int OFFSETS = STAGES * STAGE;
  static constexpr int BARS = OFFSETS + 2 * (static_cast<int>(kMaxExperts) + 1) * 4;
  static constexpr int END = BARS + (2 * STAGES + 5) * 8 + (6 + 2 * STAGES) * 4 + 1024;
  // A wide CTA takes all of an SM's TMEM and so all of its shared memory, which keeps CTAs away that
  // would wait for the first with the second in hand; narrow ones take a quarter and a half.
  static constexpr int SMEM = NARROW ? 114688 : 232448;
  static constexpr int SHARE = ACC * BM;                      // floats of a CTA's share of a split tile
  static_assert(BARS % 8 == 0 && END <= SMEM, "shared memory");
};

// Split tiles: the sums of `n` clusters before this one, at this lane's place of column 0.
struct Shares {
  const float *first;
  int n, step;
};
// 32 columns from c0 on: the accumulator and what other clusters summed before it.
__device__ __forceinline__ void add_shares(const Shares &sh, int c0, uint32_t (&r)[32]) {
  const float *from = sh.first + c0 * BM;
  for (int i = 0; i < sh.n; ++i, from += sh.step) {
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __ldcg(from + j * BM);
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + v[j]);
  }
}
__device__ __forceinline__ void read_sums(uint32_t t_acc, int c0, const Shares &sh, uint32_t (&r)[32]) {
  __syncwarp();
  tmem_ld_32x32b_x32(t_acc + c0, r);
  tmem_wait_ld();
  if (sh.n > 0) add_shares(sh, c0, r);
}
// This lane's 32 columns from c0 on for the cluster that finishes the tile.
__device__ __forceinline__ void write_share(float *to, uint32_t t_acc, int c0) {
  uint32_t r[32];
  read_sums(t_acc, c0, Shares{nullptr, 0, 0}, r);
#pragma unroll
  for (int j = 0; j < 32; ++j) __stcg(to + (c0 + j) * BM, __uint_as_float(r[j]));
}

// COUNT tokens of a feature a lane, STEP rows apart from `to` (the lane's own feature) on, the rows below
// `left` of them stored. `wide`: lanes exchange tokens for features by fours, so that each holds four
// features of every fourth token and stores 8 bytes; else one by one, which takes the memory pipe 10
// cycles a store (one GB300, 16384 rows of 16 experts, us, wide and not: 256 x 4096 46 and 78, 1024 x
// 4096 88 and 92; gated with g and u kept 1024 x 2048 105 and 127; by twos 47, 88, 108, by eights 55,
// 88, 110). By whole warps; `live`: the lane's feature exists.
template <typename T, int COUNT, int STEP>
__device__ __forceinline__ void store_tokens(T *to, int64_t ld, const float (&v)[COUNT], int left, bool live,
                                             bool wide, int lane) {
  if (!wide) {
    if (!live) return;
#pragma unroll
    for (int j = 0; j < COUNT; ++j)
      if (STEP * j < left) to[STEP * j * ld] = from_f32<T>(v[j]);
    return;
  }
  constexpr int OUT = std::is_same<T, __half>::value ? GEMM_F16 : GEMM_BF16;
  const bool one = lane & 1, two = lane & 2;
  const uint32_t pick = one ? 0x3276 : 0x5410;
  // (all exchanges before the first store: the other way round 59 us for the 46 above)
  uint32_t x[COUNT / 2];  // token 2 i + one of two features
#pragma unroll
  for (int i = 0; i < COUNT / 2; ++i) {
    const uint32_t w = pack2<OUT>(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
    x[i] = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), pick);
  }
  uint2 y[COUNT / 4];  // token 4 i + lane % 4 of four features
#pragma unroll
  for (int i = 0; i < COUNT / 4; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, two ? x[2 * i] : x[2 * i + 1], 2);
    y[i] = two ? uint2{got, x[2 * i + 1]} : uint2{x[2 * i], got};
  }
  to -= lane & 3;
#pragma unroll
  for (int i = 0; i < COUNT / 4; ++i) {
    const int row = STEP * (4 * i + (lane & 3));
    if (live && row < left) *reinterpret_cast<uint2 *>(to + row * ld) = y[i];
  }
}

// 32 tokens' columns from c0 on of this lane, the `left` first of them stored from `row` on: one
// feature f, ...
template <typename T, bool GATED, int ACC>
__device__ __forceinline__ void finish(const ExpertParams &p, uint32_t t_acc, int c0, const Shares &sh,
                                       int64_t row, int left, int64_t f, int lane) {
  uint32_t r[32], q[32];
  read_sums(t_acc, c0, sh, r);
  if (GATED) read_sums(t_acc, ACC / 2 + c0, sh, q);
  const bool live = f < p.N;
  float a[32], u[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) a[j] = __uint_as_float(r[j]);
  if (GATED) {
#pragma unroll
    for (int j = 0; j < 32; ++j) u[j] = __uint_as_float(q[j]);
    if (p.pre) {
      store_tokens<T, 32, 1>(static_cast<T *>(p.pre) + row * p.ld_pre + f, p.ld_pre, a, left, live, p.wide, lane);
      store_tokens<T, 32, 1>(static_cast<T *>(p.pre2) + row * p.ld_pre2 + f, p.ld_pre2, u, left, live, p.wide, lane);
    }
    activate_all<true>(a, p.act);
#pragma unroll
    for (int j = 0; j < 32; ++j) a[j] *= u[j];
  }
  store_tokens<T, 32, 1>(static_cast<T *>(p.C) + row * p.ldc + f, p.ldc, a, left, live, p.wide, lane);
}

// ... or g or u of one (the other 16 lanes have the other): the lower half of the warp finishes the
// even tokens, the upper half the odd ones.
template <typename T>
__device__ __forceinline__ void finish_mixed(const ExpertParams &p, uint32_t t_acc, int c0, const Shares &sh,
                                             int64_t row, int left, int64_t f, int lane) {
  uint32_t r[32];
  read_sums(t_acc, c0, sh, r);
  const bool odd = lane >= 16, gate = odd == (p.up_first != 0), live = f < p.N;
  float a[16], u[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float mine = __uint_as_float(odd ? r[2 * j + 1] : r[2 * j]);
    const float other =
        __uint_as_float(__shfl_xor_sync(0xffffffffu, odd ? r[2 * j] : r[2 * j + 1], 16));
    a[j] = gate ? mine : other;
    u[j] = gate ? other : mine;
  }
  row += odd;
  left -= odd;
  if (p.pre) {
    store_tokens<T, 16, 2>(static_cast<T *>(p.pre) + row * p.ld_pre + f, p.ld_pre, a, left, live, p.wide, lane);
    store_tokens<T, 16, 2>(static_cast<T *>(p.pre2) + row * p.ld_pre2 + f, p.ld_pre2, u, left, live, p.wide, lane);
  }
  activate_all<true>(a, p.act);
#pragma unroll
  for (int j = 0; j < 16; ++j) a[j] *= u[j];
  store_tokens<T, 16, 2>(static_cast<T *>(p.C) + row * p.ldc + f, p.ldc, a, left, live, p.wide, lane);
}

// How the tiles are shared: whole ones round-robin, or the last rounds by K-blocks. Sharing costs
// the writing and adding of sums, about `cost` K-blocks' time, and pays when it shortens the last
// round by more. With fewer tiles than clusters a tile is cut into at most sqrt(k_blocks / 4) shares,
// since their sums are added one after another.
__device__ __forceinline__ SkSchedule share_out(int tiles, int kb, int clusters, int mode, int cost, bool narrow) {
  int slots = clusters;
  if (tiles < clusters) {
    int most = 1;
    while (most < clusters && 4 * (most + 1) * (most + 1) <= kb) ++most;
    slots = min(clusters, tiles * most);
  }
  if (slots == 0) return sk_make(0, kb, clusters, 0);
  const int part = tiles < slots ? tiles : tiles % slots;  // tiles of the last round
  // K-blocks of it that a cluster is spared
  const int shared = kb < (1 << 20) ? static_cast<int>((static_cast<uint32_t>(part * kb) + slots - 1) / slots)
                                    : static_cast<int>((static_cast<int64_t>(part) * kb + slots - 1) / slots);
  const bool pays = kb - shared > cost && !(narrow && 2 * tiles > clusters);
  if (mode == 1 || part == 0 || kb < 2 || (mode != 2 && !pays)) return sk_make(tiles, kb, clusters, tiles);
  return sk_make(tiles, kb, slots, sk_dp_tiles(tiles, kb, slots, true));
}

// A cluster's pieces of work, in its order: tc::WorkIter for whole tiles as a rule, with the 64-bit
// divisions of shared ones left until there are any.
struct ExpertWork {
  SkSchedule S;
  int slot, tile;
  int64_t lo, hi;
  bool shares;
  __device__ __forceinline__ ExpertWork(const SkSchedule &s, int cluster)
      : S(s), slot(cluster), tile(cluster), lo(0), hi(0), shares(s.sk_units > 0 && cluster < s.slots) {
    if (cluster >= s.slots) tile = s.dp_tiles;
  }
  __device__ __forceinline__ bool next(SkSegment &seg) {
    if (tile < S.dp_tiles) {
      seg.tile = tile;
      seg.kb_begin = 0;
      seg.kb_end = S.kb;
      seg.role = kSegFull;
      seg.first_src = seg.last_src = -1;
      tile += S.slots;
      return true;
    }
    if (shares) {
      lo = sk_begin(S, slot);
      hi = sk_begin(S, slot + 1);
      shares = false;
    }
    if (hi <= lo) return false;
    hi = sk_segment_at(S, slot, hi, &seg);  // the share, walked from its end to its start
    return true;
  }
};

template <int MODE, bool W_MN, bool NARROW>
__global__ void __launch_bounds__(kExpertThreads, NARROW ? 2 : 1)
    expert_kernel(const __grid_constant__ ExpertMaps maps, const ExpertParams p) {
  using S = Shape<MODE, NARROW>;
  constexpr bool TWO = S::TWO;
  constexpr int ACC = S::ACC;
  constexpr int STAGES = S::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const ExpertTiles table{reinterpret_cast<int32_t *>(smem + S::OFFSETS),
                          reinterpret_cast<int32_t *>(smem + S::OFFSETS) + kMaxExperts + 1, p.experts,
                          (p.N + 2 * S::FEATURES - 1) / (2 * S::FEATURES), S::TOKENS};
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::BARS);
  uint64_t *empty = full + STAGES;
  uint64_t *tmem_full = empty + STAGES;
  uint64_t *tmem_empty = tmem_full + 2;
  uint64_t *drain = tmem_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  // Teardown words: fills this CTA's loader issued, fills the MMA issuer consumed, fills the
  // peer's loader issued, whether the other CTA aborted; then the bytes of each stage's last
  // fill, of this CTA and of the peer.
  volatile uint32_t *xs = reinterpret_cast<volatile uint32_t *>(tmem_slot + 2);
  volatile uint32_t *fill_bytes = xs + 4, *peer_bytes = fill_bytes + STAGES;

  const int warp = uniform(static_cast<int>(threadIdx.x / 32));
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], 2 * kEpi);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4 + 2 * STAGES; ++i) xs[i] = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.X[NARROW ? 0 : 3]);
    prefetch_tensormap(&maps.W);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * ACC);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  // Up to here only this CTA's own resources: the prologue may overlap the previous kernel.
  grid_dependency_wait();
  grid_launch_dependents();
  const int epoch = sk_epoch_begin(p.sk_epoch_word);
  table.fill(p.offsets, p.rows, kExpertThreads);
  __syncthreads();
  const uint32_t tmem_base = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));
  const uint32_t smem_base = smem_u32(smem);
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  const int cluster_id = blockIdx.x / 2;
  const int tiles = table.count();
  // (sums of wider tiles cost more; of the average width)
  const int width = tiles > 0 ? (table.offsets[p.experts] - table.offsets[0]) / max(tiles / table.across, 1) : 0;
  const SkSchedule sched = share_out(tiles, p.k_blocks, gridDim.x / 2, p.stream_k, 4 + width / 8, NARROW);
  const bool split = sched.dp_tiles < sched.tiles;
  // All of this CTA has read the epoch word, and the next launch reads it after this one has ended:
  // the last CTA to arrive may advance it at once.
  if (split && threadIdx.x == 32 + 1) sk_epoch_end(p.sk_epoch_word, epoch);
  __syncwarp();
  ExpertWork work(sched, cluster_id);
  SkSegment seg;

  if (warp == 0) {
    // ------------------------------------------------------ producer (both CTAs)
    // (the whole warp walks, one lane issues)
    const bool issuer = elect_one();
    uint32_t stage = 0, phase = 0, issued = 0;
    bool ok = (p.debug_flags & kDebugStallProducer) == 0;
    const int stop_after = stall_after_fills(p.debug_flags, static_cast<int>(rank));
    const uint64_t keep = l2_policy_evict_last();
    const uint32_t full_bars = mapa_shared(smem_u32(full), 0);  // the leader's
    while (ok && work.next(seg)) {
      const ExpertTiles::Tile tile = table.at(seg.tile);
      const int expert = uniform(tile.e);
      const int f0 = uniform(2 * tile.column + static_cast<int>(rank)) * S::FEATURES;
      const int half = uniform((tile.rows + 31) / 32 * 16);  // a CTA's tokens
      const int x_row = uniform(tile.row0) + static_cast<int>(rank) * half;
      // the smallest box that holds them: one copy a stage (with five 32-token ones the loader's loop
      // ran as long as four MMAs)
      const int box = NARROW ? 0 : (half - 1) / 32;
      const uint32_t bytes = static_cast<uint32_t>(S::W_ALL + kRowBytes * 32 * (box + 1));
      const int kb_end = uniform(seg.kb_end);
      for (int kb = uniform(seg.kb_begin); kb < kb_end; ++kb) {
        if (stop_after >= 0 && issued >= static_cast<uint32_t>(stop_after)) {
          ok = false;  // test hook: this loader stops here, copies still in flight
          break;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1, wd));
        if (!ok) break;
        if (issuer) {
          fill_bytes[stage] = bytes;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * bytes);
          const uint32_t w_dst = smem_base + stage * S::STAGE;
          const uint32_t fb = full_bars + stage * 8;
          const bool second = MODE == kExpertPlain && kb >= p.kb_first;
          const int k0 = (second ? kb - p.kb_first : kb) * BK;
#pragma unroll
          for (int m = 0; m < (TWO ? 2 : 1); ++m) {
            const CUtensorMap *w = (TWO ? m == 1 : second) ? &maps.W2 : &maps.W;
            const uint32_t dst = w_dst + m * W_BYTES;
            if (MODE == kExpertMixed) {
              tma_load_5d_pair(dst, w, fb, k0, 0, 0, f0 / 16, expert);
            } else if (W_MN && p.panels) {
              tma_load_4d_pair(dst, w, fb, 0, k0, f0 / 64, expert);
            } else if (W_MN) {
              tma_load_3d_pair(dst, w, fb, f0, k0, expert);
              tma_load_3d_pair(dst + PANEL_BYTES, w, fb, f0 + 64, k0, expert);
            } else {
              tma_load_3d_pair(dst, w, fb, k0, f0, expert);
            }
          }
          tma_load_2d_pair_hint(w_dst + S::W_ALL, second ? &maps.X2[box] : &maps.X[box], fb, k0, x_row, keep);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) xs[0] = issued;
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer (leader)
    if (leader) {  // (the whole warp walks, one lane issues)
      const bool issuer = elect_one();
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, consumed = 0;
      bool ok = true;
      while (ok && work.next(seg)) {
        const uint32_t n = static_cast<uint32_t>(uniform(table.at(seg.tile).rows) + 31) / 32 * 32;
        const uint32_t idesc = p.idesc | (n >> 3) << 17;
        const int blocks = uniform(seg.kb_end - seg.kb_begin);
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_empty[acc], acc_phase ^ 1, wd));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC;
        for (int i = 0; i < blocks; ++i) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, wd));
          if (!ok) break;
          ++consumed;
          tc_fence_after();
          const uint32_t w_base = smem_base + stage * S::STAGE;
          const uint64_t xd = sdesc_sw128(w_base + S::W_ALL, 16, 1024);
          const uint64_t wd_ = W_MN ? sdesc_sw128(w_base, PANEL_BYTES, 1024) : sdesc_sw128(w_base, 16, 1024);
          constexpr int W_STEP = W_MN ? 16 * kRowBytes / 16 : 32 / 16;  // 16 of K, in units of 16 bytes
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
#pragma unroll
              for (int m = 0; m < (TWO ? 2 : 1); ++m)
                mma_f16_pair(d_tmem + m * (ACC / 2), wd_ + m * (W_BYTES / 16) + kk * W_STEP,
                             xd + kk * (32 / 16), idesc, i != 0 || kk != 0);
            mma_commit_pair_multicast(&empty[stage], 0x3);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (issuer) mma_commit_pair_multicast(&tmem_full[acc], 0x3);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (issuer) {
        mma_commit_pair(drain);
        drain_wait(drain, 0, p.timeout_ns);
        xs[1] = consumed;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;
    const int half = (warp - 2) / 4;  // takes every other 32 tokens
    uint32_t acc = 0, acc_phase = 0;
    const int e = warp - 2;
    // this lane's place in a CTA's shares
    float *const place = split ? p.sk_partials + quarter * 32 + lane : nullptr;
    while (work.next(seg)) {
      const ExpertTiles::Tile tile = table.at(seg.tile);
      const int64_t f = (2 * tile.column + static_cast<int>(rank)) * S::FEATURES +
                        (MODE == kExpertMixed ? quarter * 16 + lane % 16 : quarter * 32 + lane);
      Shares sh{nullptr, 0, 2 * S::SHARE};
      bool ok = true;
      if (seg.role == kSegOwner) {
        // the clusters first_src..last_src computed the start of this tile
        for (int w = seg.first_src; ok && w <= seg.last_src; ++w)
          ok = wait_flag(p.sk_flags + (w * 2 + rank) * kEpi + e, epoch, wd);
        sh.first = place + static_cast<int64_t>(seg.first_src * 2 + static_cast<int>(rank)) * S::SHARE;
        sh.n = seg.last_src - seg.first_src + 1;
      }
      ok = ok && mbar_wait_cluster(&tmem_full[acc], acc_phase, wd);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * ACC;
      if (seg.role == kSegPartial) {
        float *to = place + static_cast<int64_t>(cluster_id * 2 + static_cast<int>(rank)) * S::SHARE;
        for (int c0 = half * 32; c0 < tile.rows; c0 += 64) {
          write_share(to, t_row, c0);
          if (TWO) write_share(to, t_row, ACC / 2 + c0);
        }
        __syncwarp();  // (every lane's stores come before the flag)
        if (lane == 0) st_release_gpu(p.sk_flags + (cluster_id * 2 + rank) * kEpi + e, epoch);
      } else {
        for (int c0 = half * 32; c0 < tile.rows; c0 += 64) {
          const int64_t row = tile.row0 + c0;
          const int left = tile.rows - c0;
          if (MODE == kExpertMixed) {
            if (p.dtype == GEMM_BF16)
              finish_mixed<__nv_bfloat16>(p, t_row, c0, sh, row, left, f, lane);
            else
              finish_mixed<__half>(p, t_row, c0, sh, row, left, f, lane);
          } else if (p.dtype == GEMM_BF16) {
            finish<__nv_bfloat16, TWO, S::ACC>(p, t_row, c0, sh, row, left, f, lane);
          } else {
            finish<__half, TWO, S::ACC>(p, t_row, c0, sh, row, left, f, lane);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_read(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    __syncwarp();
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&xs[3])), rank ^ 1u),
                          *abort_flag ? 1u : 0u);
    if (!leader) {
      st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&xs[2])), 0), xs[0]);
      for (int s = 0; s < STAGES; ++s)
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t *>(&peer_bytes[s])), 0),
                              fill_bytes[s]);
    }
  }
  tc_fence_before();
  cluster_sync();
  if (*abort_flag || xs[3]) {
    if (leader && threadIdx.x == 0)
      drain_sized_fills<STAGES>(full, xs[1], xs[0], xs[2], fill_bytes, peer_bytes, p.timeout_ns);
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * ACC);
  }
}

template <int MODE, bool W_MN, bool NARROW>
cudaError_t launch_expert(const ExpertMaps &maps, const ExpertParams &p, int grid, cudaStream_t s) {
  auto kernel = expert_kernel<MODE, W_MN, NARROW>;
  constexpr int SMEM = Shape<MODE, NARROW>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dependency_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kExpertThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

}  // namespace

cudaError_t expert_launch(ExpertMode mode, bool w_mn, bool narrow, const ExpertMaps &maps,
                          const ExpertParams &p, int grid, cudaStream_t s) {
  if (mode == kExpertTwo && !narrow)
    return w_mn ? launch_expert<kExpertTwo, true, false>(maps, p, grid, s)
                : launch_expert<kExpertTwo, false, false>(maps, p, grid, s);
  if (mode == kExpertMixed && !w_mn)
    return narrow ? launch_expert<kExpertMixed, false, true>(maps, p, grid, s)
                  : launch_expert<kExpertMixed, false, false>(maps, p, grid, s);
  if (mode != kExpertPlain) return cudaErrorInvalidValue;
  if (narrow)
    return w_mn ? launch_expert<kExpertPlain, true, true>(maps, p, grid, s)
                : launch_expert<kExpertPlain, false, true>(maps, p, grid, s);
  return w_mn ? launch_expert<kExpertPlain, true, false>(maps, p, grid, s)
              : launch_expert<kExpertPlain, false, false>(maps, p, grid, s);
}

int expert_max_clusters() {
  static std::atomic<int> cached[64];  // per device; 0 = not queried yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 1;
  }
  const int known = cached[dev].load(std::memory_order_relaxed);
  if (known > 0) return known;
  auto kernel = expert_kernel<kExpertPlain, false, false>;
  constexpr int smem = Shape<kExpertPlain, false>::SMEM;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kExpertThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int got = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&got, kernel, &cfg) != cudaSuccess || got < 1) {
    cudaGetLastError();
    return 1;
  }
  cached[dev].store(got, std::memory_order_relaxed);
  return got;
}

}  // namespace ff
}  // namespace gemm_gb300
