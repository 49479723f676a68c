// Attention calls: workspace layout and which kernels run.
#include "attention.cuh"

namespace epi {

int launch_attn_simple(const AttnArgs& a);

namespace {
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

// [counters of the decode kernel][its partial results]
size_t attn_workspace_bytes(int head_dim) {
  return round256(attn_decode_counter_bytes()) + round256(attn_decode_partial_bytes(head_dim));
}

int launch_attn(const AttnArgs& a) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  if (a.paged) {
    float* partials = reinterpret_cast<float*>(ws + round256(attn_decode_counter_bytes()));
    const int rc = launch_attn_decode(a, reinterpret_cast<uint32_t*>(ws), partials);
    if (rc != EPILORA_OK) return rc;
    if (attn_decode_takes(a.batch.max_new, a.heads / a.cache.kv_heads)) return EPILORA_OK;
  }
  return launch_attn_simple(a);
}

}  // namespace epi
