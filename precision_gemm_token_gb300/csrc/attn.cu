// Attention calls: workspace layout and which kernels run.
#include "attention.cuh"

namespace epi {

namespace {
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

// [counters of the decode kernel][of the tile kernel][partial results of the
// decode kernel][of the tile kernel]
size_t attn_workspace_bytes(int head_dim) {
  return round256(attn_decode_counter_bytes()) + round256(attn_tile_counter_bytes()) +
         round256(attn_decode_partial_bytes(head_dim)) + round256(attn_tile_partial_bytes(head_dim));
}

int launch_attn(const AttnArgs& a) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint32_t* dec_counters = reinterpret_cast<uint32_t*>(ws);
  ws += round256(attn_decode_counter_bytes());
  uint32_t* tile_counters = reinterpret_cast<uint32_t*>(ws);
  ws += round256(attn_tile_counter_bytes());
  float* dec_partials = reinterpret_cast<float*>(ws);
  float* tile_partials = reinterpret_cast<float*>(ws + round256(attn_decode_partial_bytes(a.cache.head_dim)));
  if (a.paged) {
    const int rc = launch_attn_decode(a, dec_counters, dec_partials);
    if (rc != EPILORA_OK) return rc;
    if (attn_decode_takes(a.batch.max_new, a.heads / a.cache.kv_heads)) return EPILORA_OK;
  }
  return launch_attn_tile(a, tile_counters, tile_partials);
}

}  // namespace epi
