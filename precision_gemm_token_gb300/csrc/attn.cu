// Attention calls: workspace layout and which kernels run.
#include "attention.cuh"

namespace epi {

namespace {
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

// [counters of the decode kernel][of the tile kernel][partial results of the
// decode kernel][of the tile kernel]
size_t attn_workspace_zero_bytes() { return round256(attn_decode_counter_bytes()) + round256(attn_tile_counter_bytes()); }
size_t attn_workspace_bytes(int head_dim) {
  return attn_workspace_zero_bytes() + round256(attn_decode_partial_bytes(head_dim)) +
         round256(attn_tile_partial_bytes(head_dim));
}

int launch_attn(const AttnArgs& a) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint32_t* dec_counters = reinterpret_cast<uint32_t*>(ws);
  ws += round256(attn_decode_counter_bytes());
  uint32_t* tile_counters = reinterpret_cast<uint32_t*>(ws);
  ws += round256(attn_tile_counter_bytes());
  float* dec_partials = reinterpret_cast<float*>(ws);
  float* tile_partials = reinterpret_cast<float*>(ws + round256(attn_decode_partial_bytes(a.cache.head_dim)));
  if (a.paged && attn_decode_takes(a.batch.max_new, a.heads / a.cache.kv_heads))
    return launch_attn_decode(a, dec_counters, dec_partials);
  if (!attn_tile_fits(a)) return EPILORA_ERR_UNSUPPORTED;
  // Where there are as many packed tokens as the bound allows, every sequence
  // has max_new of them and none is left for the decode kernel (or some rows are
  // padding: the tile kernel takes short sequences too). Four chunks of 37 over
  // 7999: 28.4 us behind an idle decode kernel, 24.6 us alone.
  const bool alone = !a.paged || static_cast<int64_t>(a.batch.n_seqs) * a.batch.max_new == a.batch.n_tokens;
  if (!alone) {
    const int rc = launch_attn_decode(a, dec_counters, dec_partials);
    if (rc != EPILORA_OK) return rc;
  }
  return launch_attn_tile(a, alone, tile_counters, tile_partials);
}

}  // namespace epi
