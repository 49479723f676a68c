// The rows of a mixture-of-experts batch by expert, the activations in that
// order, and the weighted sum of the experts' outputs.
//
// Few tokens are bound by latency (3 to 5 us a kernel, launch included), many by memory: of 4096 tokens with 8 of 64
// experts of 4096 x 1792 each, plan 8 us, scatter 36 (134 MB written), gather 24 (117 MB moved), sum 51 (302 MB).
#include "block_quant.cuh"

namespace epi {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kMaxExperts = EPILORA_MOE_MAX_EXPERTS;

// Counting sort of the slots by expert. A cluster of CTAs, each a run of
// slots: counts in shared memory, exchanged over the cluster; a CTA's rows of
// an expert follow those of the CTAs before it. Within a CTA the order is that
// of the additions: no result depends on it.
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const __grid_constant__ MoePlanArgs a) {
  __shared__ int count[kMaxExperts];     // this CTA's, read by the others
  __shared__ int next[kMaxExperts];      // the row of the next slot
  __shared__ int sums[kPlanThreads / 32];
  pdl_wait_primary();
  pdl_allow_dependents();
  const int n = a.tokens * a.top;
  const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  const int run = (n + ctas - 1) / ctas, first = min(run * rank, n), last = min(first + run, n);
  for (int e = threadIdx.x; e < a.experts; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  bool bad = false;
#pragma unroll 4
  for (int i = first + threadIdx.x; i < last; i += kPlanThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) atomicAdd(&count[e], 1);
    bad |= e >= a.experts;
  }
  if (bad) record_status(a.status, EPILORA_ERR_INVALID_ARG);
  cluster_arrive();
  cluster_wait();
  // exclusive sums over the experts of all CTAs' counts, a thread kPer consecutive experts
  constexpr int kPer = kMaxExperts / kPlanThreads;
  int at[kPer], total = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    at[i] = total;
    if (e < a.experts) {
      const uint32_t mine = smem_u32(&count[e]);
      for (int c = 0; c < ctas; ++c) {
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(mine, c)) : "memory");
        total += v;
        if (c < rank) at[i] += v;
      }
    }
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
      next[e] = before + at[i];
      if (rank == 0) a.plan.offsets[e] = before + at[i];
    }
  }
  if (rank == 0 && threadIdx.x == kPlanThreads - 1) a.plan.offsets[a.experts] = before + total;
  __syncthreads();
#pragma unroll 4
  for (int i = first + threadIdx.x; i < last; i += kPlanThreads) {
    const int e = a.ids[i];
    int row = -1;
    if (e >= 0 && e < a.experts) {
      row = atomicAdd(&next[e], 1);
      a.plan.slots[row] = i;
    }
    a.plan.rows[i] = row;
  }
  cluster_arrive();      // (nobody leaves while another may read its counts)
  cluster_wait();
}

struct ScatterParams {
  MoeScatterArgs a;
  int rt_log2, tiles;
};

__global__ void __launch_bounds__(kQuantThreads) moe_scatter_kernel(const __grid_constant__ ScatterParams p) {
  pdl_wait_primary();
  pdl_allow_dependents();
  const MoeScatterArgs& a = p.a;
  quant_tile<1>(static_cast<const __nv_bfloat16*>(a.q.X), a.q.M, a.q.K, a.q.ldx, a.q.Xq, a.q.scale, a.q.scale_ld, p.rt_log2,
                static_cast<int>(blockIdx.x), a.rows, a.top);
  if (a.inner == nullptr) return;
  const int n = a.q.M * a.top, nb = n_blocks(a.inner_dim);
  for (int i = static_cast<int>(blockIdx.x); i < n; i += p.tiles) {
    if (a.rows[i] >= 0) continue;
    uint4* row = reinterpret_cast<uint4*>(a.inner + static_cast<int64_t>(i) * a.inner_dim);
    for (int c = threadIdx.x; c < a.inner_dim / 16; c += kQuantThreads) row[c] = make_uint4(0, 0, 0, 0);
    for (int b = threadIdx.x; b < nb; b += kQuantThreads) a.inner_scale[static_cast<int64_t>(b) * n + i] = 0.0f;
  }
}

// A warp per slot.
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads) moe_gather_kernel(const __grid_constant__ MoeGatherArgs a) {
  pdl_wait_primary();
  pdl_allow_dependents();
  const int slot = static_cast<int>(blockIdx.x) * (kGatherThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (slot >= a.slots) return;
  // the first 2 KB of the row on their way beside the look-up
  const uint4* src = reinterpret_cast<const uint4*>(a.src + static_cast<int64_t>(slot) * a.K);
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.K / 16) v[i] = src[lane + 32 * i];
  const int row = a.rows[slot];
  if (row < 0) return;
  uint4* dst = reinterpret_cast<uint4*>(a.dst + static_cast<int64_t>(row) * a.K);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.K / 16) dst[lane + 32 * i] = v[i];
#pragma unroll 4
  for (int c = lane + 128; c < a.K / 16; c += 32) dst[c] = src[c];
  for (int b = lane; b < n_blocks(a.K); b += 32)
    a.dst_scale[static_cast<int64_t>(b) * a.slots + row] = a.src_scale[static_cast<int64_t>(b) * a.slots + slot];
}

// A CTA sums 2048 columns of one token.
constexpr int kCombineThreads = 256;
constexpr int kCombineAhead = 4;         // rows that a thread has under way

// eight consecutive parts, as they are stored
template <bool kF32>
struct Parts8 {
  uint4 v[kF32 ? 2 : 1];
};

template <bool kF32>
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
  const int64_t first = static_cast<int64_t>(t) * a.top;
  constexpr int kSize = kF32 ? 4 : 2;
  const uint8_t* parts = static_cast<const uint8_t*>(a.parts) + (first * a.hidden + n) * kSize;
  for (int j0 = 0; j0 < a.top; j0 += kCombineAhead) {
    Parts8<kF32> v[kCombineAhead];
    bool there[kCombineAhead];
#pragma unroll
    for (int q = 0; q < kCombineAhead; ++q) {
      const int e = j0 + q < a.top ? a.ids[first + j0 + q] : -1;
      there[q] = e >= 0 && e < a.experts;
      if (there[q]) {
        const uint4* src = reinterpret_cast<const uint4*>(parts + static_cast<int64_t>(j0 + q) * a.hidden * kSize);
#pragma unroll
        for (int i = 0; i < kSize / 2; ++i) v[q].v[i] = __ldcg(src + i);
      }
    }
#pragma unroll
    for (int q = 0; q < kCombineAhead; ++q) {
      if (!there[q]) continue;
      const float w = a.weights[first + j0 + q];
      alignas(16) float d[8];
      if constexpr (kF32) {
        *reinterpret_cast<Parts8<true>*>(d) = v[q];
      } else {
        unpack8(v[q].v[0], d);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(w, d[i], y[i]);
    }
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

int launch_moe_plan(const MoePlanArgs& a) {
  // one CTA counts a few thousand slots as fast as a cluster does
  const int64_t n = static_cast<int64_t>(a.tokens) * a.top;
  const unsigned ctas = n <= 4 * kPlanThreads ? 1 : 8;
  return launch_dependent(moe_plan_kernel, ctas, kPlanThreads, 0, a.stream, a, ctas);
}

int launch_moe_scatter(const MoeScatterArgs& a) {
  ScatterParams p{a, quant_rows_log2(a.q.M), 0};
  const int64_t tiles = quant_tiles(a.q.M, a.q.K, 1, p.rt_log2);
  if (tiles > 0x7fffffff) return EPILORA_ERR_UNSUPPORTED;
  p.tiles = static_cast<int>(tiles);
  return launch_dependent(moe_scatter_kernel, static_cast<unsigned>(tiles), kQuantThreads, 0, a.q.stream, p);
}

int launch_moe_gather(const MoeGatherArgs& a) {
  constexpr int per = kGatherThreads / 32;
  return launch_dependent(moe_gather_kernel, static_cast<unsigned>((a.slots + per - 1) / per), kGatherThreads, 0, a.stream, a);
}

int launch_moe_combine(const MoeCombineArgs& a) {
  const int64_t ctas = static_cast<int64_t>(a.tokens) * ((a.hidden + 8 * kCombineThreads - 1) / (8 * kCombineThreads));
  if (ctas > 0x7fffffff) return EPILORA_ERR_UNSUPPORTED;
  return launch_dependent(a.f32 ? moe_combine_kernel<true> : moe_combine_kernel<false>, static_cast<unsigned>(ctas),
                          kCombineThreads, 0, a.stream, a);
}

}  // namespace epi
