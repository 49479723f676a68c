// Shared parts of the block-scaled products: the walk over tiles, copies of
// scales, waits, tensor maps.
#pragma once
#include "block_quant.cuh"

namespace epi {

struct Tile {
  int expert, first, rows, n;      // rows [first, first + rows) of A, all of the expert's; columns' tile
};

// The tiles of a CTA in order: expert by expert, its row tiles fastest (CTAs
// next to one another then share weights in L2). Tiles of kTileRows rows.
template <bool kGrouped, int kTileRows>
struct Walk {
  const int* offsets;        // shared memory: [experts + 1]
  const int* starts;         // row tiles before each expert, [experts + 1]
  int n_tiles, M, e, total;
  __device__ Walk(int M_, int n_tiles_, int experts, const int* off, const int* st)
      : offsets(off), starts(st), n_tiles(n_tiles_), M(M_), e(0) {
    total = (kGrouped ? starts[experts] : (M + kTileRows - 1) / kTileRows) * n_tiles;
  }
  __device__ Tile at(int t) {
    Tile r;
    if (kGrouped) {
      while (starts[e + 1] * n_tiles <= t) ++e;
      const int mt = starts[e + 1] - starts[e], local = t - starts[e] * n_tiles;
      const int m = local % mt;
      r.expert = e;
      r.n = local / mt;
      r.first = offsets[e] + m * kTileRows;
      r.rows = min(kTileRows, offsets[e + 1] - r.first);
    } else {
      const int mt = total / n_tiles, m = t % mt;
      r.expert = 0;
      r.n = t / mt;
      r.first = m * kTileRows;
      r.rows = min(kTileRows, M - r.first);
    }
    return r;
  }
};

// One warp fills a walk's tables from the rows of the experts, 32 experts at a time.
template <int kTileRows>
__device__ __forceinline__ void fill_walk(const int32_t* rows_of, int experts, int* offsets, int* starts, int lane) {
  int before = 0;
  for (int e0 = 0; e0 < experts; e0 += 32) {
    const int e = e0 + lane;
    const int o0 = e <= experts ? __ldcg(rows_of + e) : 0;
    const int o1 = e < experts ? __ldcg(rows_of + e + 1) : o0;
    const int mt = (o1 - o0 + kTileRows - 1) / kTileRows;
    int sum = mt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (e < experts) {
      offsets[e] = o0;
      starts[e] = before + sum - mt;
      if (e == experts - 1) {
        offsets[e + 1] = o1;
        starts[e + 1] = before + sum;
      }
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
}

// Four bytes of global memory to shared memory; complete in order of the groups committed after them.
__device__ __forceinline__ void copy4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A wait on a barrier; gives up when it runs out (recorded) or another role of the CTA has.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_flag == 0 && mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
  if (*abort_flag == 0) {
    *abort_flag = 1;
    record_status(status, EPILORA_ERR_TIMEOUT);
  }
  return false;
}

// g / (1 + exp(-g)) within 2^-21 + |g| 2^-24 of it (the exponent's argument is rounded) down to g = -87.3; below that 0,
// where the value is less than 2^-119 (the quotient gives 0 from a divisor of 2^126 on; the formula in 32 bits does so
// from g = -88.8 on, where exp(-g) overflows). Without a division's branches: a tile's elements are all in registers, so
// this code stands there once for each of them, and has to stay in the instruction cache beside the loops.
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + exp2_approx(-1.442695041f * g)); }

// Calls with few rows (block_few.cu).
bool block_few_takes(const BlockGemmArgs& a);
int launch_block_few(const BlockGemmArgs& a);

}  // namespace epi
