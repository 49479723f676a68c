// Attention, one warp per (token, head): running maximum and sum over the
// visible positions, everything in fp32. The plain kernel the others are
// checked against.
#include "attention.cuh"
#include "ptx.cuh"

namespace epi {
namespace {

struct SimpleParams {
  AttnArgs a;
  int page_shift;
};

template <int D>
__global__ void attn_simple_kernel(const __grid_constant__ SimpleParams sp) {
  const AttnArgs& p = sp.a;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  const int h = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (h >= p.heads) return;
  int b = 0;
  for (int i = lane; i < p.batch.n_seqs; i += 32) b += __ldg(p.batch.q_start + i + 1) <= t;
  b = __reduce_add_sync(0xffffffffu, b);
  int seen = 0, first = 0;
  bool bad = false;
  if (b < p.batch.n_seqs) {
    const SeqRows s = seq_rows(p.batch.q_start, b, p.batch.n_tokens, bad);
    first = s.first;
    if (p.paged && s.n <= 16 / (p.heads / p.cache.kv_heads)) return;
    if (p.paged) {
      const int len = __ldg(p.batch.kv_len + b);
      seen = len - s.n + (t - s.first) + 1;
      if (len > (p.batch.table_pages << sp.page_shift) || s.n > p.batch.max_new) bad = true;
      seen = min(seen, p.batch.table_pages << sp.page_shift);
    } else {
      seen = t - s.first + 1;
    }
    if (t < s.first) seen = 0, bad = true;
  }
  constexpr int E = D / 32;
  float q[E], acc[E];
  const __nv_bfloat16* qr = p.q.p + t * p.q.ts + h * p.q.hs;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(qr[lane + 32 * e]), acc[e] = 0.0f;
  const int g = h / (p.heads / p.cache.kv_heads);
  const bool e4 = p.paged && p.cache.kv_fmt == EPILORA_KV_E4M3;
  const float ks = e4 ? p.cache.k_scale[g] : 1.0f, vs = e4 ? p.cache.v_scale[g] : 1.0f;
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j < seen; ++j) {
    float k[E], v[E];
    if (!p.paged) {
      const __nv_bfloat16* kr = p.k.p + (first + j) * p.k.ts + g * p.k.hs;
      const __nv_bfloat16* vr = p.v.p + (first + j) * p.v.ts + g * p.v.hs;
#pragma unroll
      for (int e = 0; e < E; ++e) k[e] = __bfloat162float(kr[lane + 32 * e]), v[e] = __bfloat162float(vr[lane + 32 * e]);
    } else {
      const int pg = __ldg(p.batch.page_table + b * p.batch.table_stride + (j >> sp.page_shift));
      const int row = j & (p.cache.page_size - 1);
      if (pg < 0 || pg >= p.cache.num_pages) {
        bad = true;
#pragma unroll
        for (int e = 0; e < E; ++e) k[e] = v[e] = 0.0f;
      } else {
        const int64_t ka = pg * p.cache.k_page_stride + g * p.cache.k_head_stride + row * p.cache.k_token_stride;
        const int64_t va = pg * p.cache.v_page_stride + g * p.cache.v_head_stride + row * p.cache.v_token_stride;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane + 32 * e;
          if (e4) {
            k[e] = e4m3_to_f32(static_cast<const uint8_t*>(p.cache.k)[ka + d]);
            v[e] = e4m3_to_f32(static_cast<const uint8_t*>(p.cache.v)[va + d]);
          } else {
            k[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.cache.k)[ka + d]);
            v[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.cache.v)[va + d]);
          }
        }
      }
    }
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += q[e] * k[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= p.scale * ks;
    const float m2 = fmaxf(m, x);
    const float c = m2 == -INFINITY ? 1.0f : expf(m - m2), w = m2 == -INFINITY ? 0.0f : expf(x - m2);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + w * v[e];
    m = m2;
  }
  if (bad && lane == 0) record_status(p.status, EPILORA_ERR_INVALID_ARG);
  __nv_bfloat16* o = p.o.p + t * p.o.ts + h * p.o.hs;
#pragma unroll
  for (int e = 0; e < E; ++e) o[lane + 32 * e] = __float2bfloat16_rn(seen > 0 ? acc[e] * vs / l : 0.0f);
  if (p.lse != nullptr && lane == 0) p.lse[static_cast<int64_t>(t) * p.heads + h] = seen > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

int launch_attn_simple(const AttnArgs& a) {
  SimpleParams p{a, a.paged ? __builtin_ctz(a.cache.page_size) : 0};
  const dim3 grid(a.batch.n_tokens, (a.heads + 3) / 4);
  if (a.cache.head_dim == 64)
    attn_simple_kernel<64><<<grid, 128, 0, a.stream>>>(p);
  else
    attn_simple_kernel<128><<<grid, 128, 0, a.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

}  // namespace epi
