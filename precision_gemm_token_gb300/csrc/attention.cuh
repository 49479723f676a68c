// Shared definitions of the attention operators: the paged key/value cache's
// append, attention over the cache, attention of packed prompts.
#pragma once
#include "common.cuh"

namespace epi {

// bf16 rows [token][head][head_dim], strides in elements
struct AttnRows {
  const __nv_bfloat16* p;
  int64_t ts, hs;
};
struct AttnOut {
  __nv_bfloat16* p;
  int64_t ts, hs;
};

struct AppendArgs {
  epilora_kv_cache cache;
  epilora_kv_batch batch;
  int heads;
  AttnRows q, k, v;
  AttnOut qo;
  const float* cos_sin;
  int n_pos, rot_dim, interleaved;
  int* status;
  cudaStream_t stream;
};
int launch_kv_append(const AppendArgs& a);

// Attention over the cache (paged != 0) or over packed prompts (k, v rows).
struct AttnArgs {
  int paged;
  epilora_kv_cache cache;   // paged; prompts: head_dim and kv_heads only
  epilora_kv_batch batch;   // prompts: n_seqs, n_tokens, q_start only
  int heads;
  AttnRows q, k, v;
  AttnOut o;
  float* lse;
  float scale;
  void* workspace;
  int* status;
  cudaStream_t stream;
};
int launch_attn(const AttnArgs& a);
size_t attn_workspace_bytes(int head_dim);
size_t attn_workspace_zero_bytes();   // of these, at the head: the counters

// A row's running maximum is raised (and its sums rescaled) only when a score
// exceeds it by this many powers of two, so that after a few tiles nothing is
// rescaled any more.
constexpr float kRaise = 8.0f;
// The weights are powers of two of the score's distance from the maximum, plus
// this: they stay below 2^(kRaise + lift), in range of the 16-bit operands. bf16
// has fp32's range. fp16 (an E4M3 cache) has most of its range above 1: with
// the maximum at 2^7 a weight is within 2^-11 of itself down to 2^-21 of the
// maximum's, and below that off by at most 2^-32 of it (without, 2^-14 and 2^-25:
// behind a few dominant positions a long context's many small weights
// vanished from the outputs, though not from the sums that divide them).
template <bool E4>
constexpr float kWeightLift = E4 ? 7.0f : 0.0f;

// attn_decode.cu: the sequences whose new tokens n satisfy
// attn_decode_takes(n, group), and the packed rows of no sequence.
__host__ __device__ inline bool attn_decode_takes(int n, int group) { return n <= 16 / group; }
int launch_attn_decode(const AttnArgs& a, uint32_t* counters, float* partials);
size_t attn_decode_counter_bytes();
size_t attn_decode_partial_bytes(int head_dim);
// attn_tile.cu: the other sequences of a call over the cache, behind the
// decode kernel; alone: all sequences of a call, over the cache or packed
// prompts, and the packed rows of none.
bool attn_tile_fits(const AttnArgs& a);   // the line's units are counted in 32 bits
int launch_attn_tile(const AttnArgs& a, bool alone, uint32_t* counters, float* partials);
size_t attn_tile_counter_bytes();
size_t attn_tile_partial_bytes(int head_dim);

// Batch metadata may be written by the previous kernel on the stream, so it is
// read with ordinary loads: the compiler takes read-only loads for invariant
// and may move them above griddepcontrol.wait.

// The new tokens of sequence b: packed rows [first, first + n), clamped to
// the packed array whatever q_start holds; `bad` is set where it had to be.
struct SeqRows {
  int first, n;
};
__device__ __forceinline__ SeqRows seq_rows(const int32_t* q_start, int b, int n_tokens, bool& bad) {
  const int s = q_start[b], e = q_start[b + 1];
  SeqRows r;
  r.first = min(max(s, 0), n_tokens);
  const int end = min(max(e, r.first), n_tokens);
  r.n = end - r.first;
  if (r.first != s || end != e || (b == 0 && s != 0)) bad = true;
  return r;
}

}  // namespace epi
