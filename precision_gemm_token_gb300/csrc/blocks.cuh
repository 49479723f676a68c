// Shared definitions of the operators in 8-bit blocks: the block quantizer,
// the block-scaled product, and the mixture-of-experts operators over it.
#pragma once
#include "common.cuh"

namespace epi {

constexpr int kBlock = 128;                      // elements of a row, and rows and columns of a weight, that share a scale
__host__ __device__ constexpr int n_blocks(int n) { return (n + kBlock - 1) / kBlock; }

// Rows of bf16 to E4M3 codes with one scale per 128 elements.
struct BlockQuantArgs {
  const void* X;
  int M, K;
  int64_t ldx;
  uint8_t* Xq;          // [M][K]
  float* scale;         // [n_blocks(K)][scale_ld]
  int64_t scale_ld;
  cudaStream_t stream;
};
int launch_block_quant(const BlockQuantArgs& a);
// A weight [N][K] with one scale per 128 x 128 block: codes [N][K], scale [n_blocks(N)][n_blocks(K)].
int launch_block_quant_weight(const void* W, int N, int K, int64_t ldw, uint8_t* Wq, float* scale, cudaStream_t stream);

// The rows of a batch by expert. Slot j of token t (number t * top + j) is
// row `row` of the sorted batch; expert e owns the rows [offsets[e], offsets[e + 1]).
struct MoePlan {
  int32_t* offsets;     // [experts + 1]
  int32_t* slots;       // row -> slot
  int32_t* rows;        // slot -> row, -1: no expert
};
struct MoePlanArgs {
  const int32_t* ids;   // [tokens][top]; outside [0, experts): no expert there
  int tokens, top, experts;
  MoePlan plan;
  int* status;
  cudaStream_t stream;
};
int launch_moe_plan(const MoePlanArgs& a);

// The activations of the slots, by row: token rows quantized and written to
// the rows of their slots (scales [n_blocks(K)][slots]). `inner`, where given,
// has zeros written for the slots without an expert.
struct MoeScatterArgs {
  BlockQuantArgs q;     // M = tokens; scale_ld = tokens * top
  int top;
  const int32_t* rows;
  uint8_t* inner;       // [tokens * top][inner_dim]
  float* inner_scale;   // [n_blocks(inner_dim)][tokens * top]
  int inner_dim;
};
int launch_moe_scatter(const MoeScatterArgs& a);

// Quantized rows by slot -> by row.
struct MoeGatherArgs {
  const uint8_t* src;
  const float* src_scale;
  uint8_t* dst;
  float* dst_scale;
  int slots, K;         // rows of both arrays, bytes of a row
  const int32_t* rows;
  cudaStream_t stream;
};
int launch_moe_gather(const MoeGatherArgs& a);

// The block-scaled product: rows of A times rows of W.
//   plain:   Y[m][n] = bf16( sum_b a_scale[b][m] w_scale[n / 128][b] sum_{k in b} A[m][k] W[n][k] ), m < M
//   grouped: the rows [offsets[e], offsets[e + 1]) times W[e]
//   gated:   grouped, W[e] is [2][N][K] (gate, up); the output is block-quantized silu(gate) * up
struct BlockGemmArgs {
  int M, N, K;          // grouped: M = rows that the arrays have
  const uint8_t* A;     // codes [M][K]
  const float* a_scale; // [n_blocks(K)][a_scale_ld]
  int64_t a_scale_ld;
  const uint8_t* W;
  const float* w_scale;
  void* Y;              // bf16 [M][ldy] (f32, grouped only: fp32)
  int64_t ldy;
  int f32, grouped, gated, experts;
  const int32_t* offsets;
  const int32_t* out_rows;   // output row of each row (NULL: the same)
  uint8_t* inner;       // gated: codes [M][N] and scales [n_blocks(N)][M]
  float* inner_scale;
  int early_weights;    // the weights may be read before the preceding kernel has finished
  int* status;
  cudaStream_t stream;
};
int launch_block_gemm(const BlockGemmArgs& a);
int block_test_late_copies();      // the test hook (epilora_test_late_block_copies)

// y[t] = bf16( sum_j weights[t][j] parts[t * top + j] ), over the slots that have an expert, in fp32
struct MoeCombineArgs {
  const int32_t* ids;
  const float* weights;
  int tokens, top, experts, hidden;
  const void* parts;    // [tokens * top][hidden], fp32 or bf16
  int f32;
  void* Y;
  int64_t ldy;
  cudaStream_t stream;
};
int launch_moe_combine(const MoeCombineArgs& a);

struct MoeRouteArgs {
  const void* logits;
  int bf16;
  int tokens, experts, top;
  int64_t ld;
  const float* bias;
  int sigmoid, groups, top_groups, group_best, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
  cudaStream_t stream;
};
int launch_moe_route(const MoeRouteArgs& a);

// A launch as a programmatic dependent of the previous kernel on the stream, in clusters of `cluster` CTAs.
template <class P>
int launch_dependent(void (*kern)(P), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, const P& p,
                     unsigned cluster = 1) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

}  // namespace epi
