// One scale per 128 elements: amax, scale and E4M3 codes of a block held by
// 16 lanes (8 elements each), as the row quantizers (quant_row.cuh) have them
// for a whole row.
#pragma once
#include "blocks.cuh"
#include "quant_row.cuh"

namespace epi {

__device__ __forceinline__ float amax8(const uint4& v) {
  float x[8];
  unpack8(v, x);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}
__device__ __forceinline__ float block_scale(float amax) { return __fdiv_rn(fmaxf(amax, kAmaxFloor), kE4M3Max); }
// x / s rounded to nearest by the corrected reciprocal product (quant_row.cuh;
// scales lie above 2^-49, the floor). An infinity in the block makes s
// infinite: with rs = 0 and 0 for s the same three operations give 0, or NaN
// for the infinity, as the division would.
struct BlockDiv {
  float s, rs;
};
__device__ __forceinline__ BlockDiv block_div(float scale) {
  return BlockDiv{isinf(scale) ? 0.0f : scale, __fdiv_rn(1.0f, scale)};
}

// One CTA's share of a quantizer grid: kQuantGroups groups of 16 lanes, each
// with kUnits blocks. The CTA covers 2^rt_log2 rows (so that the scales of
// consecutive rows are written together) by as many blocks as remain. With
// `rows`, row m goes to the rows rows[m * top] .. rows[m * top + top - 1] of
// the output (none where that is negative).
constexpr int kQuantThreads = 256;
constexpr int kQuantGroups = kQuantThreads / 16;

template <int kUnits>
__device__ __forceinline__ void quant_tile(const __nv_bfloat16* X, int M, int K, int64_t ldx,
                                           uint8_t* Xq, float* scale, int64_t scale_ld,
                                           int rt_log2, int tile, const int32_t* rows = nullptr,
                                           int top = 1) {
  const int kb = n_blocks(K);
  const int per = kUnits * kQuantGroups >> rt_log2;      // blocks of a row in a tile
  const int across = (kb + per - 1) / per;
  const int g = static_cast<int>(threadIdx.x) >> 4, lane = static_cast<int>(threadIdx.x) & 15;
  const int row = ((tile / across) << rt_log2) + (g & ((1 << rt_log2) - 1));
  const int b0 = (tile % across) * per + (g >> rt_log2);
  const int step = kQuantGroups >> rt_log2;
  const bool live = row < M;
  const __nv_bfloat16* x = X + static_cast<int64_t>(live ? row : 0) * ldx;
  uint4 v[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int k = (b0 + i * step) * kBlock + lane * 8;
    v[i] = live && k < K ? *reinterpret_cast<const uint4*>(x + k) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    float m = amax8(v[i]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int b = b0 + i * step, k = b * kBlock + lane * 8;
    const float s = block_scale(m);
    if (live && k < K) {
      const BlockDiv by = block_div(s);
      const uint2 q = quant8_e4m3_rs(v[i], by.s, by.rs);
      for (int j = 0; j < top; ++j) {
        const int to = rows == nullptr ? row : rows[static_cast<int64_t>(row) * top + j];
        if (to < 0) continue;
        *reinterpret_cast<uint2*>(Xq + static_cast<int64_t>(to) * K + k) = q;
        if (lane == 0) scale[static_cast<int64_t>(b) * scale_ld + to] = s;
      }
    }
  }
}

// Tiles of a quantizer grid, and its rows per tile: 16 where there are as
// many, fewer for a few rows (their blocks are spread over the groups then).
__host__ inline int quant_rows_log2(int M) {
  int r = 0;
  while (r < 4 && (1 << r) < M) ++r;
  return r;
}
__host__ inline int64_t quant_tiles(int M, int K, int units, int rt_log2) {
  const int per = units * kQuantGroups >> rt_log2;
  return static_cast<int64_t>((M + (1 << rt_log2) - 1) >> rt_log2) * ((n_blocks(K) + per - 1) / per);
}

}  // namespace epi
