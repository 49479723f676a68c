// Appending keys and values to the paged cache, with the position rotation of
// queries and keys on the way (epilora_kv_append).
//
//   y[a] = fl(fl(x[a] c) - fl(x[b] s)),  y[b] = fl(fl(x[b] c) + fl(x[a] s))
//
// Per token (heads + 2 kv_heads) * D bf16 elements are read once and written
// once (keys and values as bf16 or E4M3): a pure copy in bytes, bound by DRAM
// for a prefill chunk and by the chain of dependent loads (sequence ->
// position -> page and rotation row -> store) for a decode step.
//
// A block takes a token. A thread takes the same 16 elements of several head
// rows (two 16-byte loads each: for the half-split rotation the two halves of
// eight pairs), so that its cosines and sines are loaded once; three rows are on
// their way while every warp looks the token up for itself (a warp doing it for
// the block, and a barrier, took longer).
//
// Measured: 8044 tokens of 32 + 2 x 8 heads 32.3 us (6.2 TB/s), 2112 of 64 + 2 x 8
// into an E4M3 cache 20.1 to 21.6 us (4.0 TB/s, launch and first loads included),
// one token 3.1 us.
#include "attention.cuh"
#include "ptx.cuh"

namespace epi {
namespace {

struct AppendParams {
  epilora_kv_cache c;
  epilora_kv_batch b;
  int rows;   // heads + 2 kv_heads (kv rows only: no Q)
  AttnRows q, k, v;
  AttnOut qo;
  const float* cos_sin;
  int n_pos, rot_dim, interleaved;
  int page_shift;
  int* status;
};

// Sequence of packed row t: the number of sequences that end at or before t
// (n_seqs: none holds t). One warp counts together; sequences without new
// tokens count like any other.
__device__ __forceinline__ int find_seq(const int32_t* q_start, int n_seqs, int t, int lane) {
  int n = 0;
  for (int i = lane; i < n_seqs; i += 32) n += q_start[i + 1] <= t;
  return __reduce_add_sync(0xffffffffu, n);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = cvt_e4m3x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

constexpr int kThreads = 128;
// rows of a thread under way: 34.2, 32.3, 32.7, 41.1 us with 2, 3, 4, 5 for 8044 tokens of 48 rows, 21.0, 20.1 to 21.6,
// 21.8, 22.7 us for 2112 tokens of 80 rows into an E4M3 cache (with seven blocks per SM bf16 spills from five on, E4M3
// 92, 164, 356 bytes with three, four, five)
constexpr int kBatch = 3;

template <int D, bool E4>
__global__ void __launch_bounds__(kThreads, 7) kv_append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait_primary();
  constexpr int kPerRow = D / 16, kRowStep = kThreads / kPerRow;
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int u = threadIdx.x % kPerRow, r0 = threadIdx.x / kPerRow;
  const int half = p.rot_dim >> 1;
  const bool rotated = p.cos_sin != nullptr && u < p.rot_dim / 16;    // of a q or k row
  const bool split = p.interleaved == 0;
  const int kvh = p.c.kv_heads, nq = p.rows - 2 * kvh;
  // element offsets of the two groups of eight; of a rotated row
  const int e0 = u * 16, e1 = e0 + 8;
  const int f0 = rotated && split ? u * 8 : e0, f1 = rotated && split ? half + u * 8 : e1;

  bool looked_up = false, live = false;
  int64_t k_at = 0, v_at = 0;
  float c[8], s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;

#pragma unroll 1
  for (int rb = 0; rb < p.rows; rb += kBatch * kRowStep) {
    uint4 v[kBatch][2];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = rb + r0 + y * kRowStep;
      v[y][0] = v[y][1] = make_uint4(0, 0, 0, 0);
      if (r < p.rows) {
        const int h = r < nq ? r : (r < nq + kvh ? r - nq : r - nq - kvh);
        const AttnRows& src = r < nq ? p.q : (r < nq + kvh ? p.k : p.v);
        const __nv_bfloat16* row = src.p + t * src.ts + h * src.hs;
        v[y][0] = *reinterpret_cast<const uint4*>(row + (r < nq + kvh ? f0 : e0));
        v[y][1] = *reinterpret_cast<const uint4*>(row + (r < nq + kvh ? f1 : e1));
      }
    }
    if (!looked_up) {
      looked_up = true;
      bool bad = false;
      const int b = find_seq(p.b.q_start, p.b.n_seqs, t, lane);
      if (b < p.b.n_seqs) {
        const SeqRows q = seq_rows(p.b.q_start, b, p.b.n_tokens, bad);
        const int pos = p.b.kv_len[b] - q.n + (t - q.first);
        const int at = pos >> p.page_shift;
        if (t < q.first || q.n > p.b.max_new) bad = true;
        if (!bad && pos >= 0) {
          if (at >= p.b.table_pages || (p.cos_sin != nullptr && pos >= p.n_pos)) {
            bad = true;
          } else {
            const int page = p.b.page_table[b * p.b.table_stride + at];
            if (rotated) {
              const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.rot_dim + u * 8;
#pragma unroll
              for (int j = 0; j < 8; j += 4) {
                const float4 cv = *reinterpret_cast<const float4*>(row + j);
                const float4 sv = *reinterpret_cast<const float4*>(row + half + j);
                c[j] = cv.x, c[j + 1] = cv.y, c[j + 2] = cv.z, c[j + 3] = cv.w;
                s[j] = sv.x, s[j + 1] = sv.y, s[j + 2] = sv.z, s[j + 3] = sv.w;
              }
            }
            const int64_t row = pos & (p.c.page_size - 1);
            if (page < 0 || page >= p.c.num_pages) {
              bad = true;
            } else {
              k_at = page * p.c.k_page_stride + row * p.c.k_token_stride;
              v_at = page * p.c.v_page_stride + row * p.c.v_token_stride;
              live = true;
            }
          }
        }
      }
      if (bad && threadIdx.x == 0) record_status(p.status, EPILORA_ERR_INVALID_ARG);
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = rb + r0 + y * kRowStep;
      if (r >= p.rows) break;
      const int kind = r < nq ? 0 : (r < nq + kvh ? 1 : 2);
      const int h = kind == 0 ? r : (kind == 1 ? r - nq : r - nq - kvh);
      const int o0 = kind != 2 ? f0 : e0, o1 = kind != 2 ? f1 : e1;
      if (kind == 0 && !live) v[y][0] = v[y][1] = make_uint4(0, 0, 0, 0);
      if (kind != 0 && !live) continue;
      float x0[8], x1[8];
      const bool codes = E4 && kind != 0;
      if ((rotated && kind != 2) || codes) {
        unpack8(v[y][0], x0);
        unpack8(v[y][1], x1);
      }
      if (rotated && kind != 2 && live) {
        if (split) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float a = x0[j], b = x1[j];
            x0[j] = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
            x1[j] = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a = x0[2 * j], b = x0[2 * j + 1];
            x0[2 * j] = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
            x0[2 * j + 1] = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
            a = x1[2 * j], b = x1[2 * j + 1];
            x1[2 * j] = __fsub_rn(__fmul_rn(a, c[j + 4]), __fmul_rn(b, s[j + 4]));
            x1[2 * j + 1] = __fadd_rn(__fmul_rn(b, c[j + 4]), __fmul_rn(a, s[j + 4]));
          }
        }
        if (!codes) v[y][0] = pack8(x0), v[y][1] = pack8(x1);
      }
      if (codes) {
        const float scale = (kind == 1 ? p.c.k_scale : p.c.v_scale)[h];
        uint8_t* o = kind == 1 ? static_cast<uint8_t*>(p.c.k) + k_at + h * p.c.k_head_stride
                               : static_cast<uint8_t*>(p.c.v) + v_at + h * p.c.v_head_stride;
        *reinterpret_cast<uint2*>(o + o0) = codes8(x0, scale);
        *reinterpret_cast<uint2*>(o + o1) = codes8(x1, scale);
      } else {
        __nv_bfloat16* o = kind == 0   ? p.qo.p + t * p.qo.ts + h * p.qo.hs
                           : kind == 1 ? static_cast<__nv_bfloat16*>(p.c.k) + k_at + h * p.c.k_head_stride
                                       : static_cast<__nv_bfloat16*>(p.c.v) + v_at + h * p.c.v_head_stride;
        *reinterpret_cast<uint4*>(o + o0) = v[y][0];
        *reinterpret_cast<uint4*>(o + o1) = v[y][1];
      }
    }
  }
}

}  // namespace

int launch_kv_append(const AppendArgs& a) {
  AppendParams p{};
  p.c = a.cache;
  p.b = a.batch;
  p.rows = (a.qo.p != nullptr ? a.heads : 0) + 2 * a.cache.kv_heads;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.qo = a.qo;
  p.cos_sin = a.cos_sin;
  p.n_pos = a.n_pos;
  p.rot_dim = a.rot_dim;
  p.interleaved = a.interleaved;
  p.page_shift = __builtin_ctz(a.cache.page_size);
  p.status = a.status;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.batch.n_tokens, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool e4 = a.cache.kv_fmt == EPILORA_KV_E4M3;
  auto kern = a.cache.head_dim == 64 ? (e4 ? kv_append_kernel<64, true> : kv_append_kernel<64, false>)
                                     : (e4 ? kv_append_kernel<128, true> : kv_append_kernel<128, false>);
  const cudaError_t rc = cudaLaunchKernelEx(&cfg, kern, p);
  return rc == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

}  // namespace epi
