// The rows of a mixture-of-experts batch by expert, with the quantization of
// the activations beside it, and the weighted sum of the experts' outputs.
#include "block_quant.cuh"

namespace epi {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kMaxExperts = EPILORA_MOE_MAX_EXPERTS;

// Offsets and rows by counting; one CTA. The order of the rows of an expert
// is the order of the additions: no result depends on it.
__device__ void plan_block(const MoePrepArgs& a) {
  __shared__ int count[kMaxExperts];
  __shared__ int sums[kPlanThreads / 32];
  const int n = a.tokens * a.top;
  for (int e = threadIdx.x; e < a.experts; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) atomicAdd(&count[e], 1);
    if (e >= a.experts) bad = true;
  }
  if (bad) record_status(a.status, EPILORA_ERR_INVALID_ARG);
  __syncthreads();
  // exclusive sums: each thread kMaxExperts / kPlanThreads consecutive experts
  constexpr int kPer = kMaxExperts / kPlanThreads;
  int mine[kPer], total = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    mine[i] = total;
    total += e < a.experts ? count[e] : 0;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) sums[warp] = before;
  before -= total;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < a.experts) {
      count[e] = before + mine[i];
      a.plan.offsets[e] = before + mine[i];
      if (e == a.experts - 1) a.plan.offsets[a.experts] = before + total;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) a.plan.rows[atomicAdd(&count[e], 1)] = i;
  }
}

struct PrepParams {
  MoePrepArgs a;
  int rt_log2, tiles;
};

// CTA 0 the plan, the others the quantizer's tiles and then the slots that
// have no expert.
__global__ void __launch_bounds__(kPlanThreads) moe_prep_kernel(const __grid_constant__ PrepParams p) {
  pdl_wait_primary();
  pdl_allow_dependents();
  if (blockIdx.x == 0) {
    plan_block(p.a);
    return;
  }
  const MoePrepArgs& a = p.a;
  quant_tile<1>(static_cast<const __nv_bfloat16*>(a.q.X), a.q.M, a.q.K, a.q.ldx, a.q.Xq, a.q.scale, a.q.scale_ld,
                p.rt_log2, static_cast<int>(blockIdx.x) - 1);
  const int n = a.tokens * a.top, nb = n_blocks(a.inner_dim);
  for (int i = static_cast<int>(blockIdx.x) - 1; i < n; i += p.tiles) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) continue;
    uint4* row = reinterpret_cast<uint4*>(a.inner + static_cast<int64_t>(i) * a.inner_dim);
    for (int c = threadIdx.x; c < a.inner_dim / 16; c += kPlanThreads) row[c] = make_uint4(0, 0, 0, 0);
    for (int b = threadIdx.x; b < nb; b += kPlanThreads) a.inner_scale[static_cast<int64_t>(b) * n + i] = 0.0f;
  }
}

// A CTA sums 2048 columns of one token.
constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(const __grid_constant__ MoeCombineArgs a) {
  pdl_wait_primary();
  pdl_allow_dependents();
  const int across = (a.hidden + 8 * kCombineThreads - 1) / (8 * kCombineThreads);
  const int t = static_cast<int>(blockIdx.x) / across;
  const int n = (static_cast<int>(blockIdx.x) % across) * 8 * kCombineThreads + static_cast<int>(threadIdx.x) * 8;
  if (n >= a.hidden) return;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.0f;
  for (int j = 0; j < a.top; ++j) {
    const int64_t slot = static_cast<int64_t>(t) * a.top + j;
    const int e = a.ids[slot];
    if (e < 0 || e >= a.experts) continue;
    const float w = a.weights[slot];
    float d[8];
    unpack8(__ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.parts) + slot * a.hidden + n)), d);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(w, d[i], y[i]);
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) + t * a.ldy + n) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace

int launch_moe_prep(const MoePrepArgs& a) {
  PrepParams p{a, 0, 0};
  if (a.quant) {
    p.rt_log2 = quant_rows_log2(a.q.M);
    const int64_t tiles = quant_tiles(a.q.M, a.q.K, 1, p.rt_log2);
    if (tiles >= 0x7fffffff) return EPILORA_ERR_UNSUPPORTED;
    p.tiles = static_cast<int>(tiles);
  }
  return launch_dependent(moe_prep_kernel, static_cast<unsigned>(p.tiles + 1), kPlanThreads, 0, a.stream, p);
}

int launch_moe_combine(const MoeCombineArgs& a) {
  const int64_t ctas = static_cast<int64_t>(a.tokens) * ((a.hidden + 8 * kCombineThreads - 1) / (8 * kCombineThreads));
  if (ctas > 0x7fffffff) return EPILORA_ERR_UNSUPPORTED;
  return launch_dependent(moe_combine_kernel, static_cast<unsigned>(ctas), kCombineThreads, 0, a.stream, a);
}

}  // namespace epi
