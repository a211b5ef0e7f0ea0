// expert_tiles.cuh -- what the experts' product kernels share: the walk over the tiles of all
// experts, whose row counts are known on the device only, and the end of a CTA pair's pipeline
// after an abort.
#pragma once

#include "tc_common.cuh"

namespace gemm_gb300 {
namespace ff {

// Copies offsets (at most kMaxExperts + 1) to shared memory, kept inside [0, rows]. A walk takes
// them in order and never back, so that offsets that decrease leave an expert without rows
// instead of sending it outside.
__device__ __forceinline__ void load_offsets(int32_t *to, const int32_t *offsets, int experts,
                                             int rows, int threads) {
  for (int e = threadIdx.x; e <= experts; e += threads) to[e] = max(0, min(offsets[e], rows));
}

// Experts in order with their tiles: `lines` tiles along the rows (of `width` rows each, the last
// one shorter) times `across` tiles the other way. Tiles are numbered through all experts.
struct ExpertWalk {
  const int32_t *offsets;
  int experts, across, most, step;  // most: rows a tile, at most; step: width's granularity
  int e, lo, hi, begin, count, lines, width;
  __device__ __forceinline__ ExpertWalk(const int32_t *o, int n, int a, int m, int s)
      : offsets(o), experts(n), across(a), most(m), step(s), e(-1), lo(0), hi(o[0]), begin(0), count(0),
        lines(0), width(0) {}
  // Advances to the expert of tile t (t grows from call to call); false past the last one.
  __device__ __forceinline__ bool seek(int t) {
    while (t >= begin + count) {
      if (++e >= experts) return false;
      begin += count;
      lo = hi;
      hi = max(lo, offsets[e + 1]);
      const int n = hi - lo;
      lines = (n + most - 1) / most;
      // rows shared evenly: 300 rows of 256 at most are 160 and 140, not 256 and 44
      width = lines > 0 ? ((n + lines - 1) / lines + step - 1) / step * step : 0;
      count = lines * across;
    }
    return true;
  }
  // Line and column of tile t of the expert found: lines run fastest, in groups of eight, so that
  // neighbouring tiles share both operands through L2.
  __device__ __forceinline__ void place(int t, int &line, int &column) const {
    int i = t - begin, first = 0, n = lines;
    if (lines > 8) {
      const int group = i / (8 * across);
      first = group * 8;
      i -= group * 8 * across;
      n = min(lines - first, 8);
    }
    column = i / n;
    line = first + (i - column * n);
  }
};

// tc::drain_pair_fills for fills of different sizes: bytes[s] and peer_bytes[s] are those of the
// last fill of stage s that this CTA and the peer issued.
template <int STAGES>
__device__ __noinline__ void drain_sized_fills(uint64_t *full, uint32_t consumed,
                                               uint32_t leader_issued, uint32_t peer_issued,
                                               const volatile uint32_t *bytes,
                                               const volatile uint32_t *peer_bytes,
                                               uint64_t timeout_ns) {
  const uint32_t end = leader_issued > peer_issued ? leader_issued : peer_issued;
  for (uint32_t i = consumed; i < end; ++i) {
    uint64_t *bar = &full[i % STAGES];
    if (i >= leader_issued)
      mbar_arrive_expect_tx(bar, peer_bytes[i % STAGES]);  // only the peer issued this fill
    else if (i >= peer_issued)
      mbar_complete_tx(bar, bytes[i % STAGES]);  // the peer's part of this fill never comes
    tc::drain_wait(bar, (i / STAGES) & 1, timeout_ns);
  }
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z, int32_t w, int32_t v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

}  // namespace ff
}  // namespace gemm_gb300
