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
// A thread takes 16 elements of a head row at a time (two 16-byte loads: for
// the half-split rotation the two halves of eight pairs). A few tokens get a
// block each, one unit a thread; many are taken four to a block with four units
// a thread under way. Either way the first rows are on their way while a warp
// per token looks the token up.
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

// what the look-up of a token leaves
struct Token {
  int64_t k_at, v_at;   // cache offsets of its row, head 0
  int pos;              // < 0: nothing is appended
};

// TB tokens per block, BATCH units per thread under way
template <int TB, int BATCH, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ Token tokens[TB];
  pdl_wait_primary();
  const int t0 = blockIdx.x * TB;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = p.c.head_dim / 16, per_token = p.rows * per_row;
  const int total = min(TB, p.b.n_tokens - t0) * per_token;
  const int half = p.rot_dim >> 1;
  const int rot_units = p.cos_sin != nullptr ? p.rot_dim / 16 : 0;
  const bool split = p.interleaved == 0;
  const int kvh = p.c.kv_heads, nq = p.rows - 2 * kvh;

  // unit i of the block: token, tensor (0 q, 1 k, 2 v), head, unit of the row
  struct Unit {
    int tok, kind, h, u, e0, e1;
    bool rot;
  };
  auto unit_of = [&](int i) {
    Unit x;
    x.tok = 0;
#pragma unroll
    for (int k = 1; k < TB; ++k)
      if (i >= per_token) i -= per_token, ++x.tok;
    const int r = i / per_row;
    x.u = i - r * per_row;
    x.kind = r < nq ? 0 : (r < nq + kvh ? 1 : 2);
    x.h = x.kind == 0 ? r : (x.kind == 1 ? r - nq : r - nq - kvh);
    x.rot = x.u < rot_units && x.kind != 2;
    // element offsets of the two groups of eight
    x.e0 = x.rot && split ? x.u * 8 : x.u * 16;
    x.e1 = x.rot && split ? half + x.u * 8 : x.u * 16 + 8;
    return x;
  };

  bool looked_up = false;
  for (int i0 = threadIdx.x; i0 - static_cast<int>(threadIdx.x) < total; i0 += blockDim.x * BATCH) {
    uint4 v[BATCH][2];
#pragma unroll
    for (int y = 0; y < BATCH; ++y) {
      const int i = i0 + y * blockDim.x;
      v[y][0] = v[y][1] = make_uint4(0, 0, 0, 0);
      if (i < total) {
        const Unit x = unit_of(i);
        const AttnRows& src = x.kind == 0 ? p.q : (x.kind == 1 ? p.k : p.v);
        const __nv_bfloat16* row = src.p + static_cast<int64_t>(t0 + x.tok) * src.ts + x.h * src.hs;
        v[y][0] = *reinterpret_cast<const uint4*>(row + x.e0);
        v[y][1] = *reinterpret_cast<const uint4*>(row + x.e1);
      }
    }
    if (!looked_up) {
      looked_up = true;
      for (int k = warp; k < TB; k += blockDim.x >> 5) {
        const int t = t0 + k;
        Token tk{0, 0, -1};
        bool bad = false;
        const int b = t < p.b.n_tokens ? find_seq(p.b.q_start, p.b.n_seqs, t, lane) : p.b.n_seqs;
        if (b < p.b.n_seqs) {
          const SeqRows s = seq_rows(p.b.q_start, b, p.b.n_tokens, bad);
          const int pos = p.b.kv_len[b] - s.n + (t - s.first);
          const int at = pos >> p.page_shift;
          if (t < s.first || s.n > p.b.max_new) bad = true;
          if (!bad && pos >= 0) {
            if (at >= p.b.table_pages || (rot_units > 0 && pos >= p.n_pos)) {
              bad = true;
            } else {
              const int page = p.b.page_table[b * p.b.table_stride + at];
              const int64_t row = pos & (p.c.page_size - 1);
              if (page < 0 || page >= p.c.num_pages) {
                bad = true;
              } else {
                tk.k_at = page * p.c.k_page_stride + row * p.c.k_token_stride;
                tk.v_at = page * p.c.v_page_stride + row * p.c.v_token_stride;
                tk.pos = pos;
              }
            }
          }
        }
        if (lane == 0) {
          tokens[k] = tk;
          if (bad) record_status(p.status, EPILORA_ERR_INVALID_ARG);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int y = 0; y < BATCH; ++y) {
      const int i = i0 + y * blockDim.x;
      if (i >= total) break;
      const Unit x = unit_of(i);
      const Token tk = tokens[x.tok];
      const bool live = tk.pos >= 0;
      float x0[8], x1[8];
      unpack8(v[y][0], x0);
      unpack8(v[y][1], x1);
      if (live && x.rot) {
        const float* row = p.cos_sin + static_cast<int64_t>(tk.pos) * p.rot_dim + x.u * 8;
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
        v[y][0] = pack8(x0);
        v[y][1] = pack8(x1);
      }
      if (x.kind == 0) {
        __nv_bfloat16* o = p.qo.p + static_cast<int64_t>(t0 + x.tok) * p.qo.ts + x.h * p.qo.hs;
        const uint4 z = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(o + x.e0) = live ? v[y][0] : z;
        *reinterpret_cast<uint4*>(o + x.e1) = live ? v[y][1] : z;
      } else if (live) {
        const bool is_k = x.kind == 1;
        const int64_t at = is_k ? tk.k_at + x.h * p.c.k_head_stride : tk.v_at + x.h * p.c.v_head_stride;
        if (p.c.kv_fmt == EPILORA_KV_BF16) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(is_k ? p.c.k : p.c.v) + at;
          *reinterpret_cast<uint4*>(o + x.e0) = v[y][0];
          *reinterpret_cast<uint4*>(o + x.e1) = v[y][1];
        } else {
          uint8_t* o = static_cast<uint8_t*>(is_k ? p.c.k : p.c.v) + at;
          const float s = (is_k ? p.c.k_scale : p.c.v_scale)[x.h];
          *reinterpret_cast<uint2*>(o + x.e0) = codes8(x0, s);
          *reinterpret_cast<uint2*>(o + x.e1) = codes8(x1, s);
        }
      }
    }
  }
}

// Tokens from which on a block takes four: with fewer the blocks of one token
// each fill the SMs at once.
constexpr int kManyTokens = 512;

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
  const bool many = a.batch.n_tokens >= kManyTokens;
  int threads = 256;
  if (!many) {
    const int rounds = (units + 1023) / 1024;
    threads = ((units + rounds - 1) / rounds + 31) / 32 * 32;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(many ? (a.batch.n_tokens + 3) / 4 : a.batch.n_tokens, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t rc = many ? cudaLaunchKernelEx(&cfg, kv_append_kernel<4, 4, 256>, p)
                              : cudaLaunchKernelEx(&cfg, kv_append_kernel<1, 1, 1024>, p);
  return rc == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

}  // namespace epi
