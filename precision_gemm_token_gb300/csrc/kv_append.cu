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
// One thread block per token, one thread per 16 elements of a head row (two
// 16-byte loads: for the half-split rotation the two halves of eight pairs).
// Every thread starts its loads of the row before it looks the token up, so
// that the look-up chain runs behind them.
#include "attention.cuh"
#include "ptx.cuh"

namespace epi {
namespace {

struct AppendParams {
  epilora_kv_cache c;
  epilora_kv_batch b;
  int heads, rows;   // rows = heads + 2 kv_heads (kv rows only: no Q)
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

__global__ void __launch_bounds__(1024) kv_append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait_primary();
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int units = p.c.head_dim / 16;
  const int total = p.rows * units;
  const int half = p.rot_dim >> 1;
  const int rot_units = p.cos_sin != nullptr ? p.rot_dim / 16 : 0;
  const bool split = p.interleaved == 0;
  bool known = false;
  int pos = -1;
  bool live = false;
  int64_t page = 0;
  int row_in_page = 0;
  // whole warps go round together (find_seq wants all 32 lanes)
  const int rounds = (total + blockDim.x - 1) / blockDim.x;
  for (int it = 0; it < rounds; ++it) {
    const int i = it * blockDim.x + threadIdx.x;
    const bool mine = i < total;
    const int r = mine ? i / units : 0;
    const int u = mine ? i - r * units : 0;
    // which tensor the row belongs to
    const int kvh = p.c.kv_heads;
    const int nq = p.rows - 2 * kvh;
    const int kind = r < nq ? 0 : (r < nq + kvh ? 1 : 2);
    const int h = kind == 0 ? r : (kind == 1 ? r - nq : r - nq - kvh);
    const bool rot = u < rot_units && kind != 2;
    // element offsets of the two groups of eight
    const int e0 = rot && split ? u * 8 : u * 16;
    const int e1 = rot && split ? half + u * 8 : u * 16 + 8;
    const AttnRows& src = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (mine) {
      const __nv_bfloat16* x = src.p + t * src.ts + h * src.hs;
      v0 = *reinterpret_cast<const uint4*>(x + e0);
      v1 = *reinterpret_cast<const uint4*>(x + e1);
    }
    if (!known) {
      known = true;
      const int b = find_seq(p.b.q_start, p.b.n_seqs, t, lane);
      if (b < p.b.n_seqs) {
        bool bad = false;
        const SeqRows s = seq_rows(p.b.q_start, b, p.b.n_tokens, bad);
        const int len = p.b.kv_len[b];
        pos = len - s.n + (t - s.first);
        const int at = pos >> p.page_shift;
        row_in_page = pos & (p.c.page_size - 1);
        if (t < s.first || s.n > p.b.max_new) bad = true;
        if (!bad && pos >= 0) {
          if (at >= p.b.table_pages || (rot_units > 0 && pos >= p.n_pos)) {
            bad = true;
          } else {
            const int pg = p.b.page_table[b * p.b.table_stride + at];
            if (pg < 0 || pg >= p.c.num_pages)
              bad = true;
            else
              page = pg, live = true;
          }
        }
        if (bad && threadIdx.x == 0) record_status(p.status, EPILORA_ERR_INVALID_ARG);
      }
    }
    if (!mine) continue;
    float x0[8], x1[8];
    unpack8(v0, x0);
    unpack8(v1, x1);
    if (live && rot) {
      const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.rot_dim + u * 8;
      float c[8], s[8];
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const float4 cv = *reinterpret_cast<const float4*>(row + j);
        const float4 sv = *reinterpret_cast<const float4*>(row + half + j);
        c[j] = cv.x, c[j + 1] = cv.y, c[j + 2] = cv.z, c[j + 3] = cv.w;
        s[j] = sv.x, s[j + 1] = sv.y, s[j + 2] = sv.z, s[j + 3] = sv.w;
      }
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
      v0 = pack8(x0);
      v1 = pack8(x1);
    }
    if (kind == 0) {
      __nv_bfloat16* o = p.qo.p + t * p.qo.ts + h * p.qo.hs;
      const uint4 z = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(o + e0) = live ? v0 : z;
      *reinterpret_cast<uint4*>(o + e1) = live ? v1 : z;
    } else if (live) {
      const bool is_k = kind == 1;
      const int64_t at = page * (is_k ? p.c.k_page_stride : p.c.v_page_stride) +
                         h * (is_k ? p.c.k_head_stride : p.c.v_head_stride) +
                         row_in_page * (is_k ? p.c.k_token_stride : p.c.v_token_stride);
      if (p.c.kv_fmt == EPILORA_KV_BF16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(is_k ? p.c.k : p.c.v) + at;
        *reinterpret_cast<uint4*>(o + e0) = v0;
        *reinterpret_cast<uint4*>(o + e1) = v1;
      } else {
        uint8_t* o = static_cast<uint8_t*>(is_k ? p.c.k : p.c.v) + at;
        const float s = (is_k ? p.c.k_scale : p.c.v_scale)[h];
        *reinterpret_cast<uint2*>(o + e0) = codes8(x0, s);
        *reinterpret_cast<uint2*>(o + e1) = codes8(x1, s);
      }
    }
  }
}

}  // namespace

int launch_kv_append(const AppendArgs& a) {
  AppendParams p{};
  p.c = a.cache;
  p.b = a.batch;
  p.heads = a.heads;
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
  const int units = p.rows * (a.cache.head_dim / 16);
  const int rounds = (units + 1023) / 1024;
  const int threads = ((units + rounds - 1) / rounds + 31) / 32 * 32;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.batch.n_tokens, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append_kernel, p) == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

}  // namespace epi
