// expert_tiles.cuh -- what the experts' product kernels share: the walk over the tiles of all
// experts, whose row counts are known on the device only, and the end of a CTA pair's pipeline
// after an abort.
#pragma once

#include "tc_common.cuh"

namespace gemm_gb300 {
namespace ff {

// The tiles of all experts, numbered through: an expert with n rows has ceil(n / most) tiles along
// its rows times `across` the other way. Both tables live in shared memory: the experts' first rows
// (experts + 1) and first tiles (experts + 1; the last one is the number of tiles).
struct ExpertTiles {
  int32_t *offsets, *begins;
  int experts, across;
  int most;  // rows a tile, at most: a power of two

  // Fills the tables from the caller's offsets, by all threads; a barrier has to follow. Offsets are
  // kept inside [0, rows] and never decrease, so that no row has two experts and none lies outside.
  __device__ __forceinline__ void fill(const int32_t *from, int rows, int threads) const {
    for (int e = threadIdx.x; e <= experts; e += threads) offsets[e] = max(0, min(from[e], rows));
    __syncthreads();
    if (threadIdx.x >= 32) return;
    int high = offsets[0], sum = 0;
    __syncwarp();
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int e = e0 + static_cast<int>(threadIdx.x);
      int end = e < experts ? offsets[e + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, end, d);
        if (static_cast<int>(threadIdx.x) >= d) end = max(end, v);
      }
      end = max(end, high);
      int start = __shfl_up_sync(0xffffffffu, end, 1);
      if (threadIdx.x == 0) start = high;
      const int mine = e < experts ? (end - start + most - 1) / most * across : 0;
      int through = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, through, d);
        if (static_cast<int>(threadIdx.x) >= d) through += v;
      }
      if (e < experts) {
        offsets[e + 1] = end;
        begins[e] = sum + through - mine;
        if (e == experts - 1) begins[experts] = sum + through;
      }
      high = __shfl_sync(0xffffffffu, end, 31);
      sum += __shfl_sync(0xffffffffu, through, 31);
    }
  }
  __device__ __forceinline__ int count() const { return begins[experts]; }

  struct Tile {
    int e, row0, rows, column;
  };
  // Tile t: its rows are an even share of the expert's, in steps of 32 (594 rows of 256 at most are
  // 224, 192 and 178, not 256, 256 and 82). Tiles along the rows run fastest, in groups of eight, so that
  // neighbours share both operands through L2.
  __device__ __forceinline__ Tile at(int t) const {
    int lo = 0, hi = experts;  // begins[lo] <= t < begins[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (begins[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int first_row = offsets[lo], n = offsets[lo + 1] - first_row;
    const int lines = (n + most - 1) / most;
    const int steps = (n + 31) / 32, share = lines == 1 ? steps : steps / lines, extra = steps - share * lines;
    int i = t - begins[lo], first = 0, group = lines;
    if (lines > 8) {
      const int g = i / (8 * across);
      first = g * 8;
      i -= g * 8 * across;
      group = min(lines - first, 8);
    }
    Tile tile;
    tile.e = lo;
    tile.column = group == 1 ? i : i / group;
    const int line = first + (i - tile.column * group);
    const int row = 32 * (line * share + min(line, extra));
    tile.row0 = first_row + row;
    tile.rows = min(32 * (share + (line < extra ? 1 : 0)), n - row);
    return tile;
  }
};

// The same in every lane, and known to be: the tensor core's instructions take their operands from
// uniform registers, and moving each there from a lane's own costs the issuing thread some 20 cycles
// an operand. With whole warps walking the loop, one elected lane issuing, and the values that come
// from shared memory passed through this, four MMAs and their commit take 165 cycles to issue
// instead of 350 (measured), less than the 512 they run.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// Tells the MMA issuer of the pair that this warp has read an accumulator. The reads are complete
// (tcgen05.wait::ld) and no other memory is handed over, so that nothing has to be released: at
// cluster scope a release waits for the warp's stores of the tile, some 3000 cycles when memory is
// busy, and held up the next tile's MMAs (weight gradients of 256 rows an expert, 4096 x 2048: 252 us
// against 307).
__device__ __forceinline__ void arrive_read(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

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
