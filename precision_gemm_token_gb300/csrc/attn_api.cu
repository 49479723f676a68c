// C ABI of the attention operators: argument validation.
#include <cmath>

#include "attention.cuh"

using namespace epi;

namespace {

inline bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a strided tensor of rows [token][head][head_dim]
bool rows_ok(const void* p, int64_t ts, int64_t hs, int tokens, int heads, int head_dim) {
  if (p == nullptr || !al(p, 16)) return false;
  if (ts % 8 != 0 || hs % 8 != 0 || ts < 0 || hs < 0) return false;
  // a head's elements overlap neither the next head's nor the next token's
  if (heads > 1 && hs < head_dim) return false;
  if (tokens > 1 && ts < head_dim) return false;
  return true;
}

bool heads_ok(int heads, int kv_heads, int head_dim) {
  return kv_heads >= 1 && heads >= 1 && heads % kv_heads == 0 && heads <= 65536 && head_dim >= 1;
}

// the kernels count a sequence's (token, head) rows in 31 bits
bool rows_fit(int tokens, int heads) { return static_cast<int64_t>(tokens) * heads < (int64_t{1} << 30); }

int cache_check(const epilora_kv_cache* c, int heads) {
  if (c == nullptr || c->reserved != 0) return EPILORA_ERR_INVALID_ARG;
  if (c->kv_fmt != EPILORA_KV_BF16 && c->kv_fmt != EPILORA_KV_E4M3) return EPILORA_ERR_INVALID_ARG;
  if (!heads_ok(heads, c->kv_heads, c->head_dim)) return EPILORA_ERR_INVALID_ARG;
  if (c->page_size < 1 || c->num_pages < 1) return EPILORA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return EPILORA_ERR_UNSUPPORTED;
  if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size < 16 || c->page_size > 256)
    return EPILORA_ERR_UNSUPPORTED;
  if (c->k == nullptr || c->v == nullptr || !al(c->k, 16) || !al(c->v, 16)) return EPILORA_ERR_INVALID_ARG;
  const int64_t unit = c->kv_fmt == EPILORA_KV_BF16 ? 8 : 16;   // elements of 16 bytes
  const int64_t strides[6] = {c->k_page_stride, c->k_head_stride, c->k_token_stride,
                              c->v_page_stride, c->v_head_stride, c->v_token_stride};
  for (int i = 0; i < 6; ++i) {
    if (strides[i] % unit != 0 || strides[i] < c->head_dim) return EPILORA_ERR_INVALID_ARG;
    // (a tensor map's stride stays below 2^40 bytes)
    if (strides[i] >= (int64_t{1} << 38)) return EPILORA_ERR_UNSUPPORTED;
  }
  if (c->kv_fmt == EPILORA_KV_E4M3 &&
      (c->k_scale == nullptr || c->v_scale == nullptr || !al(c->k_scale, 4) || !al(c->v_scale, 4)))
    return EPILORA_ERR_INVALID_ARG;
  return EPILORA_OK;
}

int batch_check(const epilora_kv_batch* b, int page_size) {
  if (b == nullptr || b->n_seqs < 0 || b->n_tokens < 0 || b->max_new < 0) return EPILORA_ERR_INVALID_ARG;
  if (b->n_tokens == 0) return EPILORA_OK;
  if (b->table_pages < 0 || b->table_stride < b->table_pages) return EPILORA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(b->table_pages) * page_size > (int64_t{1} << 30)) return EPILORA_ERR_UNSUPPORTED;
  if (b->q_start == nullptr || !al(b->q_start, 4)) return EPILORA_ERR_INVALID_ARG;
  if (b->n_seqs > 0 && (b->kv_len == nullptr || !al(b->kv_len, 4))) return EPILORA_ERR_INVALID_ARG;
  if (b->n_seqs > 0 && b->table_pages > 0 && (b->page_table == nullptr || !al(b->page_table, 4)))
    return EPILORA_ERR_INVALID_ARG;
  return EPILORA_OK;
}

int workspace_check(int head_dim, const void* ws, size_t bytes) {
  return ws == nullptr || !al(ws, 256) || bytes < attn_workspace_bytes(head_dim) ? EPILORA_ERR_WORKSPACE : EPILORA_OK;
}

inline AttnRows rows(const void* p, int64_t ts, int64_t hs) {
  return AttnRows{static_cast<const __nv_bfloat16*>(p), ts, hs};
}
inline AttnOut out_rows(void* p, int64_t ts, int64_t hs) { return AttnOut{static_cast<__nv_bfloat16*>(p), ts, hs}; }

}  // namespace

extern "C" {

EPILORA_API int epilora_kv_append(const epilora_kv_cache* cache, const epilora_kv_batch* batch, int heads,
                                  const void* Q, int64_t q_token_stride, int64_t q_head_stride, const void* K,
                                  int64_t k_token_stride, int64_t k_head_stride, const void* V,
                                  int64_t v_token_stride, int64_t v_head_stride, const float* cos_sin, int n_pos,
                                  int rot_dim, int interleaved, void* Qout, int64_t qo_token_stride,
                                  int64_t qo_head_stride, int* status_dev, void* stream) {
  int rc = cache_check(cache, heads);
  if (rc == EPILORA_OK) rc = batch_check(batch, cache->page_size);
  if (rc != EPILORA_OK) return rc;
  if (cos_sin != nullptr &&
      (!al(cos_sin, 16) || n_pos < 0 || rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > cache->head_dim))
    return EPILORA_ERR_INVALID_ARG;
  const int T = batch->n_tokens, D = cache->head_dim;
  if (T == 0) return EPILORA_OK;
  if ((Q == nullptr) != (Qout == nullptr) || (Q == nullptr && cos_sin != nullptr)) return EPILORA_ERR_INVALID_ARG;
  if (Q != nullptr && (!rows_ok(Q, q_token_stride, q_head_stride, T, heads, D) ||
                       !rows_ok(Qout, qo_token_stride, qo_head_stride, T, heads, D)))
    return EPILORA_ERR_INVALID_ARG;
  if (Q != nullptr && Q == Qout && (q_token_stride != qo_token_stride || q_head_stride != qo_head_stride))
    return EPILORA_ERR_INVALID_ARG;
  if (!rows_ok(K, k_token_stride, k_head_stride, T, cache->kv_heads, D) ||
      !rows_ok(V, v_token_stride, v_head_stride, T, cache->kv_heads, D))
    return EPILORA_ERR_INVALID_ARG;
  AppendArgs a{};
  a.cache = *cache;
  a.batch = *batch;
  a.heads = heads;
  a.q = rows(Q, q_token_stride, q_head_stride);
  a.k = rows(K, k_token_stride, k_head_stride);
  a.v = rows(V, v_token_stride, v_head_stride);
  a.qo = out_rows(Qout, qo_token_stride, qo_head_stride);
  a.cos_sin = cos_sin;
  a.n_pos = n_pos;
  a.rot_dim = cos_sin != nullptr ? rot_dim : 0;
  a.interleaved = interleaved != 0;
  a.status = status_dev;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_kv_append(a);
}

EPILORA_API size_t epilora_attention_workspace_bytes(int head_dim) {
  return head_dim == 64 || head_dim == 128 ? attn_workspace_bytes(head_dim) : 0;
}

EPILORA_API size_t epilora_attention_workspace_zero_bytes(void) { return attn_workspace_zero_bytes(); }

EPILORA_API int epilora_paged_attention(const epilora_kv_cache* cache, const epilora_kv_batch* batch, int heads,
                                        const void* Q, int64_t q_token_stride, int64_t q_head_stride, float scale,
                                        void* O, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                                        void* workspace, size_t workspace_bytes, int* status_dev, void* stream) {
  int rc = cache_check(cache, heads);
  if (rc == EPILORA_OK) rc = batch_check(batch, cache->page_size);
  if (rc != EPILORA_OK) return rc;
  if (!std::isfinite(scale)) return EPILORA_ERR_INVALID_ARG;
  const int T = batch->n_tokens, D = cache->head_dim;
  if (T == 0) return EPILORA_OK;
  if (!rows_fit(T, heads)) return EPILORA_ERR_UNSUPPORTED;
  if (!rows_ok(Q, q_token_stride, q_head_stride, T, heads, D) ||
      !rows_ok(O, o_token_stride, o_head_stride, T, heads, D) || !al(lse, 4))
    return EPILORA_ERR_INVALID_ARG;
  rc = workspace_check(D, workspace, workspace_bytes);
  if (rc != EPILORA_OK) return rc;
  AttnArgs a{};
  a.paged = 1;
  a.cache = *cache;
  a.batch = *batch;
  a.heads = heads;
  a.q = rows(Q, q_token_stride, q_head_stride);
  a.o = out_rows(O, o_token_stride, o_head_stride);
  a.lse = lse;
  a.scale = scale;
  a.workspace = workspace;
  a.status = status_dev;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attn(a);
}

EPILORA_API int epilora_prompt_attention(int n_seqs, int n_tokens, const int32_t* q_start, int heads, int kv_heads,
                                         int head_dim, const void* Q, int64_t q_token_stride, int64_t q_head_stride,
                                         const void* K, int64_t k_token_stride, int64_t k_head_stride, const void* V,
                                         int64_t v_token_stride, int64_t v_head_stride, float scale, void* O,
                                         int64_t o_token_stride, int64_t o_head_stride, float* lse, void* workspace,
                                         size_t workspace_bytes, int* status_dev, void* stream) {
  if (n_seqs < 0 || n_tokens < 0 || !heads_ok(heads, kv_heads, head_dim) || !std::isfinite(scale))
    return EPILORA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return EPILORA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return EPILORA_OK;
  if (!rows_fit(n_tokens, heads)) return EPILORA_ERR_UNSUPPORTED;
  if (q_start == nullptr || !al(q_start, 4)) return EPILORA_ERR_INVALID_ARG;
  if (!rows_ok(Q, q_token_stride, q_head_stride, n_tokens, heads, head_dim) ||
      !rows_ok(K, k_token_stride, k_head_stride, n_tokens, kv_heads, head_dim) ||
      !rows_ok(V, v_token_stride, v_head_stride, n_tokens, kv_heads, head_dim) ||
      !rows_ok(O, o_token_stride, o_head_stride, n_tokens, heads, head_dim) || !al(lse, 4))
    return EPILORA_ERR_INVALID_ARG;
  const int rc = workspace_check(head_dim, workspace, workspace_bytes);
  if (rc != EPILORA_OK) return rc;
  AttnArgs a{};
  a.cache.kv_heads = kv_heads;
  a.cache.head_dim = head_dim;
  a.batch.n_seqs = n_seqs;
  a.batch.n_tokens = n_tokens;
  a.batch.max_new = n_tokens;
  a.batch.q_start = q_start;
  a.heads = heads;
  a.q = rows(Q, q_token_stride, q_head_stride);
  a.k = rows(K, k_token_stride, k_head_stride);
  a.v = rows(V, v_token_stride, v_head_stride);
  a.o = out_rows(O, o_token_stride, o_head_stride);
  a.lse = lse;
  a.scale = scale;
  a.workspace = workspace;
  a.status = status_dev;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attn(a);
}

}  // extern "C"
