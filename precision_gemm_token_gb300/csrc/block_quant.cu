// Block quantizers: rows of activations with one scale per 128 elements, and
// (at load time) weights with one per 128 x 128 block.
//
//   s = fl32(max(amax, 1e-12) / 448),  code = E4M3(fl32(x / s))
//
// Bound: memory (2 bytes read and 1 written per element): 8192 x 14336 in 64.6 us, 5.5 TB/s, 81 % of the copy rate
// (four blocks a group of 16 lanes, six CTAs per SM; 69 us at four or five, 75 and 71 with 2 and 8 blocks a group).
#include "block_quant.cuh"

namespace epi {

namespace {

struct QuantParams {
  const __nv_bfloat16* X;
  uint8_t* Xq;
  float* scale;
  int64_t ldx, scale_ld;
  int M, K, rt_log2;
};

template <int kUnits>
__global__ void __launch_bounds__(kQuantThreads, 6) block_quant_kernel(const __grid_constant__ QuantParams p) {
  pdl_wait_primary();
  pdl_allow_dependents();
  quant_tile<kUnits>(p.X, p.M, p.K, p.ldx, p.Xq, p.scale, p.scale_ld, p.rt_log2, static_cast<int>(blockIdx.x));
}

struct QuantWeightParams {
  const __nv_bfloat16* W;
  uint8_t* Wq;
  float* scale;
  int64_t ldw;
  int N, K;
};

// One CTA per 128 x 128 block: 16 groups of 16 lanes, 8 rows a group.
__global__ void __launch_bounds__(kQuantThreads) block_quant_weight_kernel(const __grid_constant__ QuantWeightParams p) {
  __shared__ float red[kQuantThreads / 32];
  pdl_wait_primary();
  const int kb = n_blocks(p.K);
  const int nb = static_cast<int>(blockIdx.x) / kb, b = static_cast<int>(blockIdx.x) % kb;
  const int g = static_cast<int>(threadIdx.x) >> 4, lane = static_cast<int>(threadIdx.x) & 15;
  const int k = b * kBlock + lane * 8;
  uint4 v[8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * kBlock + g + i * kQuantGroups;
    v[i] = n < p.N && k < p.K ? *reinterpret_cast<const uint4*>(p.W + n * p.ldw + k) : make_uint4(0, 0, 0, 0);
    m = fmaxf(m, amax8(v[i]));
  }
  const float s = block_scale(block_max(m, red));
  const BlockDiv by = block_div(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * kBlock + g + i * kQuantGroups;
    if (n < p.N && k < p.K)
      *reinterpret_cast<uint2*>(p.Wq + static_cast<int64_t>(n) * p.K + k) =
          quant8_e4m3_rs(v[i], by.s, by.rs);
  }
  if (threadIdx.x == 0) p.scale[static_cast<int64_t>(nb) * kb + b] = s;
}

}  // namespace

int launch_block_quant(const BlockQuantArgs& a) {
  QuantParams p{static_cast<const __nv_bfloat16*>(a.X), a.Xq, a.scale, a.ldx, a.scale_ld, a.M, a.K, quant_rows_log2(a.M)};
  // four blocks a group (four loads under way per thread) once that still fills the SMs
  const int64_t t4 = quant_tiles(a.M, a.K, 4, p.rt_log2);
  if (t4 >= 2 * num_sms()) {
    if (t4 > 0x7fffffff) return EPILORA_ERR_UNSUPPORTED;
    return launch_dependent(block_quant_kernel<4>, static_cast<unsigned>(t4), kQuantThreads, 0, a.stream, p);
  }
  return launch_dependent(block_quant_kernel<1>, static_cast<unsigned>(quant_tiles(a.M, a.K, 1, p.rt_log2)),
                          kQuantThreads, 0, a.stream, p);
}

int launch_block_quant_weight(const void* W, int N, int K, int64_t ldw, uint8_t* Wq, float* scale,
                              cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(n_blocks(N)) * n_blocks(K);
  if (blocks > 0x7fffffff) return EPILORA_ERR_UNSUPPORTED;
  QuantWeightParams p{static_cast<const __nv_bfloat16*>(W), Wq, scale, ldw, N, K};
  return launch_dependent(block_quant_weight_kernel, static_cast<unsigned>(blocks), kQuantThreads, 0, stream, p);
}

}  // namespace epi
