// Attention of chunks of new tokens over the paged cache, and of whole packed
// prompts, on the tensor cores (tcgen05).
//
//   S = Q K^T,  P = exp2(c S - c m),  O += P V,  l += sum P,  c = scale log2 e
//
// The rows of a key/value head are its group's heads of consecutive new
// tokens (row = token * G + head), cut into tiles of 2 x 128; the keys and
// values into tiles of 128 positions. Per row tile and position tile the two
// products are 4 x 128 x 128 x head_dim fused multiply-adds, 2048 cycles of
// the SM's tensor pipe at head_dim 128, against 2 x 128 x 128 exponentials:
// the tensor pipe bounds it as long as the softmax of one half runs while the
// products of the other half do.
//
// One thread block per SM, twelve warps (sixteen for an E4M3 cache):
//   0-3, 4-7  two softmax groups, one per 128 rows ("stream"): a thread owns a
//             row, reads its scores from TMEM, keeps the row's maximum and
//             sum in registers, writes the weights back over the scores
//             (16-bit, the A operand of the second product) and, where the
//             maximum rose by more than 2^8, rescales the row of O in TMEM
//   8         walks the block's pieces of work and tells them to the others;
//             copies queries, and key and value tiles into a ring of shared
//             memory, by TMA
//   9         issues the products; S and O of both streams fill the TMEM
//   10        bf16: cleans the value rows that some row must not see
//   11        issues every other copy of the tiles (with pages of 16 positions
//             a bf16 tile takes 16; one warp alone: 185 us instead of 164 for a
//             chunk of 2048 over 4096, 64 heads)
//   12-15     E4M3: convert the copied codes to fp16 tiles
// Where an item has at most 128 rows both streams take the same rows and
// alternate the position tiles; they meet at the end.
//
// The position tiles of all (sequence, head, row tile) items form one line
// that is split evenly over the blocks, whatever the lengths; an item cut
// between blocks is joined by the block that finishes last, in the order of
// the pieces.
//
// Measured (heads of 128): a prompt of 8192, 64 / 8 heads, 686 to 731 us by card
// (1600 to 1500 TFLOP/s); 16 prompts of up to 1024, 32 / 8 heads, 102 us (605, an
// item's fixed costs); 512 new tokens over 16300, E4M3, 101 us (1180: a step of
// both streams takes some 3500 cycles, the products 2048 of them, the conversion
// of its two tiles beside them 2200; the rest is not accounted for).
#include "attention.cuh"
#include "ptx.cuh"

namespace epi {
namespace {

// registers per thread of the softmax warps and of the others, within the
// block's at launch; the softmax keeps 64 scores and 16 packed weights in
// registers (in the launch's 168 it spills, more than the L1 left beside the
// ring holds)
template <bool E4>
struct TileWarps {
  static constexpr int kThreads = E4 ? 512 : 384;
  static constexpr int kLaunch = E4 ? 128 : 168, kSoftmax = E4 ? 192 : 208, kOther = E4 ? 64 : 88;
  static_assert(256 * kSoftmax + (kThreads - 256) * kOther <= kThreads * kLaunch, "split of the block's registers");
};
constexpr int kPosTile = 128;      // positions per tile
constexpr int kRowTile = 128;      // rows per stream
constexpr int kItemRows = 2 * kRowTile;
constexpr int kTileMaxCtas = 512;
constexpr int kGroups = 256;       // entries of the block's table of sequence weights
// cost of an item besides its tiles, in tiles (2, 3, 4 on one card: a prompt of 8192, 64 heads 707, 686, 699 us; 16
// prompts of at most 1024 101, 103, 105 us; four chunks of 37 over 7999, then behind the decode kernel, 29.5, 28.4, 27.7 us)
constexpr int kItemCost = 3;
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

constexpr int kPieces = 4;         // pieces of work told ahead
constexpr int kPieceInts = 16;

template <int D, bool E4>
struct TileCfg {
  static constexpr int kTileBytes = kPosTile * D * 2;            // 16-bit key or value tile
  static constexpr int kBlock = 128 * 128;                       // 128 rows of 64 elements, swizzled
  static constexpr int kQBytes = 2 * kTileBytes;
  // 160 KB of tiles: five 32 KB ones at head_dim 128. E4M3 at 128: four 16-bit tiles and two of codes (with
  // three and four, the next keys' tile is free only when this step's values are done, and so converted late)
  static constexpr int kStages = (E4 ? 128 : 160) * 1024 / kTileBytes;
  static constexpr int kRawBytes = kPosTile * D;                 // E4M3 codes of a tile
  static constexpr int kRawStages = E4 ? 32 * 1024 / kRawBytes : 0;
  static constexpr int kRing = kQBytes, kRaw = kRing + kStages * kTileBytes;
  static constexpr int kPlan = kRaw + kRawStages * kRawBytes;
  static constexpr int kBars = kPlan + kGroups * 4;
  // barriers: three per stage, two per raw stage, 24 more; then 12 words of flags
  static constexpr int kBarBytes = (3 * kStages + 2 * kRawStages + 24) * 8 + 12 * 4;
  static constexpr int kPieceAt = kBars + (kBarBytes + 15) / 16 * 16;
  static constexpr int kBytes = kPieceAt + kPieces * kPieceInts * 4;
  static constexpr int kSmem = 1024 + kBytes;
  static_assert(kSmem <= 232448, "shared memory of a block");
};

struct TileParams {
  CUtensorMap tk, tv, tq;
  int q_tma;               // queries are copied by TMA (see q_boxes_fit)
  epilora_kv_batch b;
  epilora_kv_cache c;      // paged
  AttnRows q, k, v;        // k, v: prompts
  AttnOut o;
  float* lse;
  int paged;
  int alone;               // no decode kernel before this one: every sequence is taken
  int heads, kv_heads, group;
  uint32_t group_mul;      // row / group = row * group_mul >> group_shift for rows below 2^30
  int group_shift;
  int page_shift;
  int box_rows;            // rows per TMA box
  int o_sectors;           // every output row is 32-byte aligned
  float scale;
  uint32_t* counters;      // [2 gridDim.x], zero between calls
  float4* partials;        // [2 gridDim.x][(2 + D) * 256 / 4]
  int* status;
};

// row / group by a multiplication (the walk divides often; a division by a
// number the compiler does not know is some thirty instructions each time):
// group_mul = 2^(31 + s) / group rounded up, s = ceil(log2 group), is off by less
// than one, which moves the quotient by less than 2^30 / 2^(31 + s) < 1 / group.
__device__ __forceinline__ int token_of(const TileParams& p, int row) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(row)) * p.group_mul) >> p.group_shift);
}

struct TileSeq {
  int first, n, len, base, rts;   // packed rows, tokens held, position of new token 0, row tiles (0: not of the class)
};
__device__ __forceinline__ TileSeq tile_seq(const TileParams& p, int b, bool& bad) {
  TileSeq s;
  const SeqRows r = seq_rows(p.b.q_start, b, p.b.n_tokens, bad);
  s.first = r.first;
  s.n = r.n;
  if (p.paged) {
    const int len = p.b.kv_len[b];
    const int cap = p.b.table_pages << p.page_shift;
    if (len > cap || len < 0 || r.n > p.b.max_new) bad = true;
    s.base = len - r.n;
    s.len = max(min(len, cap), 0);
    s.rts = !p.alone && attn_decode_takes(r.n, p.group) ? 0 : (r.n * p.group + kItemRows - 1) / kItemRows;
  } else {
    s.base = 0;
    s.len = r.n;
    s.rts = (r.n * p.group + kItemRows - 1) / kItemRows;
  }
  return s;
}
// positions that row `row` of the sequence sees
__device__ __forceinline__ int row_sees(const TileParams& p, const TileSeq& s, int row) {
  return max(min(s.base + token_of(p, row) + 1, s.len), 0);
}
__device__ __forceinline__ int item_tiles(const TileParams& p, const TileSeq& s, int rt) {
  const int e = row_sees(p, s, min((rt + 1) * kItemRows, s.n * p.group) - 1);
  return max((e + kPosTile - 1) / kPosTile, 1);
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The line: every item takes item_tiles units, after kItemCost units that
// stand for what an item costs besides its tiles (queries, the first tile's
// maximum, the output); a piece is a run of units of one item.
// units of all row tiles of a sequence, one key/value head (whole warp)
__device__ __forceinline__ uint32_t seq_weight(const TileParams& p, int b, int lane, bool& bad) {
  const TileSeq s = tile_seq(p, b, bad);
  uint32_t w = 0;
  for (int rt = lane; rt < s.rts; rt += 32) w += kItemCost + item_tiles(p, s, rt);
  return __reduce_add_sync(0xffffffffu, w);
}

// Walks the pieces of a thread block's range of the line (one warp).
struct TileWalk {
  uint32_t x, end;     // units still to do
  uint32_t each, more; // units per block: each + 1 for the first `more` blocks, else each
  int b, h, rt;
  TileSeq s;
  int nt;              // tiles of the item
  int u0, u1;          // this piece's units of it
  uint32_t item0;      // line position of the item's first unit
  __device__ __forceinline__ uint32_t start_of(uint32_t cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ uint32_t owner_of(uint32_t unit) const {
    const uint32_t low = more * (each + 1);
    return unit < low ? unit / (each + 1) : more + (unit - low) / each;
  }
};

__device__ __forceinline__ void tile_piece(TileWalk& w) {
  w.u0 = static_cast<int>(w.x - w.item0);
  w.u1 = static_cast<int>(min(static_cast<uint32_t>(kItemCost + w.nt - w.u0), w.end - w.x)) + w.u0;
}

// The table of sequence weights, by the whole block.
__device__ __forceinline__ void tile_plan(const TileParams& p, uint32_t* plan, int warp, int warps, int lane) {
  const int per = (p.b.n_seqs + kGroups - 1) / kGroups;     // sequences per table entry
  const int entries = per == 0 ? 0 : (p.b.n_seqs + per - 1) / per;
  bool bad = false;
  for (int e = warp; e < entries; e += warps) {
    uint32_t v = 0;
    for (int b = e * per; b < min((e + 1) * per, p.b.n_seqs); ++b) v += seq_weight(p, b, lane, bad);
    if (lane == 0) plan[e] = v;
  }
  if (bad && blockIdx.x == 0) record_status(p.status, EPILORA_ERR_INVALID_ARG);
  __syncthreads();
}

// One warp; false: nothing to do.
__device__ __forceinline__ bool tile_begin(const TileParams& p, TileWalk& w, const uint32_t* plan, int lane) {
  const int per = (p.b.n_seqs + kGroups - 1) / kGroups;
  const int entries = per == 0 ? 0 : (p.b.n_seqs + per - 1) / per;
  bool bad = false;
  constexpr int kMine = kGroups / 32;
  uint32_t mine[kMine], sum = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int e = lane * kMine + i;
    mine[i] = e < entries ? plan[e] * p.kv_heads : 0;
    sum += mine[i];
  }
  const uint32_t inc = warp_scan(sum, lane);
  const uint32_t total = __shfl_sync(0xffffffffu, inc, 31);
  const uint32_t ctas = min(gridDim.x, total);
  if (blockIdx.x >= ctas) return false;
  w.each = total / ctas;
  w.more = total - w.each * ctas;
  w.x = w.start_of(blockIdx.x);
  w.end = w.start_of(blockIdx.x + 1);
  // the table entry that holds x
  const uint32_t hit = __ballot_sync(0xffffffffu, inc > w.x);
  const int l = __ffs(hit) - 1;
  uint32_t at = inc - sum;
  int e = lane * kMine;
#pragma unroll
  for (int i = 0; i < kMine - 1; ++i)
    if (at + mine[i] <= w.x && e == lane * kMine + i) at += mine[i], ++e;
  at = __shfl_sync(0xffffffffu, at, l);
  e = __shfl_sync(0xffffffffu, e, l);
  // the sequence in it
  uint32_t weight = 0;
  int b = e * per;
  for (;; ++b) {
    if (b >= p.b.n_seqs) return false;   // metadata changed under the call
    weight = seq_weight(p, b, lane, bad);
    if (at + weight * p.kv_heads > w.x) break;
    at += weight * p.kv_heads;
  }
  w.b = b;
  w.s = tile_seq(p, b, bad);
  w.h = static_cast<int>((w.x - at) / weight);
  at += w.h * weight;
  // the row tile
  for (int r0 = 0;; r0 += 32) {
    if (r0 >= w.s.rts) return false;
    const uint32_t c = r0 + lane < w.s.rts ? kItemCost + item_tiles(p, w.s, r0 + lane) : 0;
    const uint32_t in = warp_scan(c, lane);
    const uint32_t found = __ballot_sync(0xffffffffu, at + in > w.x);
    if (found != 0) {
      const int k = __ffs(found) - 1;
      w.rt = r0 + k;
      w.nt = static_cast<int>(__shfl_sync(0xffffffffu, c, k)) - kItemCost;
      w.item0 = at + __shfl_sync(0xffffffffu, in - c, k);
      break;
    }
    at += __shfl_sync(0xffffffffu, in, 31);
  }
  tile_piece(w);
  return true;
}

__device__ __forceinline__ bool tile_next(const TileParams& p, TileWalk& w) {
  w.x += w.u1 - w.u0;
  if (w.x >= w.end) return false;
  w.item0 += kItemCost + w.nt;
  if (++w.rt == w.s.rts) {
    w.rt = 0;
    if (++w.h == p.kv_heads) {
      w.h = 0;
      bool bad = false;
      do {   // x < end: a sequence of the class follows
        if (++w.b >= p.b.n_seqs) return false;
        w.s = tile_seq(p, w.b, bad);
      } while (w.s.rts == 0);
    }
  }
  w.nt = item_tiles(p, w.s, w.rt);
  tile_piece(w);
  return true;
}

// A piece as the walking warp tells it to the other roles.
struct Piece {
  int b, h;            // sequence, key/value head
  int first, base, len;
  int row0, rows;      // of the sequence's (token, head) rows
  int see_all;         // positions every row sees
  int see_end;         // positions the last row sees
  int t0, t1;          // position tiles; t0 == t1: no more work
  int whole;           // the item's only piece
  int first_cta, pieces;   // of an item in several pieces: the blocks first_cta, ...
  int slot, slot0;     // where this piece's, and the first piece's, partial result goes
  // two row tiles; else both streams share one
  __device__ __forceinline__ bool two() const { return rows > kRowTile; }
};
static_assert(sizeof(Piece) == kPieceInts * 4, "one int per field");

__device__ __forceinline__ void piece_of(const TileParams& p, const TileWalk& w, Piece& q) {
  q.b = w.b;
  q.h = w.h;
  q.first = w.s.first;
  q.base = w.s.base;
  q.len = w.s.len;
  q.row0 = w.rt * kItemRows;
  q.rows = min(kItemRows, w.s.n * p.group - q.row0);
  q.see_all = row_sees(p, w.s, q.row0);
  q.see_end = row_sees(p, w.s, q.row0 + q.rows - 1);
  q.t0 = max(w.u0 - kItemCost, 0);
  q.t1 = max(w.u1 - kItemCost, 0);
  q.whole = q.t0 == 0 && q.t1 == w.nt;
  q.first_cta = q.pieces = q.slot = q.slot0 = 0;
  if (q.whole) return;
  // the blocks that hold the item's first and last tile
  const uint32_t tile0 = w.item0 + kItemCost;
  q.first_cta = static_cast<int>(w.owner_of(tile0));
  q.pieces = static_cast<int>(w.owner_of(tile0 + w.nt - 1)) - q.first_cta + 1;
  // a piece that starts its block's range goes to the block's slot 0, the one that ends it to slot 1
  q.slot = 2 * blockIdx.x + (w.x == w.start_of(blockIdx.x) ? 0 : 1);
  q.slot0 = 2 * q.first_cta + (w.start_of(q.first_cta) >= w.item0 ? 0 : 1);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the registers of a TMEM load are read from here on
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

// whether a 32-bit word of two bf16 holds a NaN or an infinity
__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t v) {
  return ((v & 0x7F80u) == 0x7F80u) | ((v & 0x7F800000u) == 0x7F800000u);
}
// whether a 32-bit word of four E4M3 codes holds a NaN (they have no infinity)
__device__ __forceinline__ bool e4m3x4_nan(uint32_t v) {
  return (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}
// four E4M3 codes with the NaN among them replaced by zero
__device__ __forceinline__ uint32_t e4m3x4_strip_nan(uint32_t v) {
#pragma unroll
  for (int z = 0; z < 32; z += 8)
    if (((v >> z) & 0x7Fu) == 0x7Fu) v &= ~(0xFFu << z);
  return v;
}

// One tile of scores to weights; a thread owns a row, m is in units of S, the
// row sees columns below lim. A row's first tile is read for its maximum
// first. After that the weights of each half (64 columns) are taken against
// the maximum so far while the half's own is being found; only where it is
// more than kRaise above (hardly ever) is the row of O rescaled, after the
// products already under way, and the half taken again. The weights go over
// scores already read; `ready` tells the products' warp of each half, `half_in`
// waits until the first half's product is in O.
template <int D, bool E4, typename Ready, typename HalfIn>
__device__ __forceinline__ bool softmax_tile(uint32_t ts, uint32_t to, float c, int lim, bool started, float& m,
                                             float& l, Ready ready, HalfIn half_in) {
  // (Loops are kept rolled where their body is long enough: unrolled, the
  // kernel's paths evict one another from the instruction cache.)
  if (__any_sync(0xffffffffu, lim < kPosTile)) {
    // scores that the row must not see
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      const int n = lim - 32 * g;
      if (__all_sync(0xffffffffu, n >= 32)) continue;
      const uint32_t seen = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
      uint32_t v[32];
      tmem_ld_32x32b_x32(ts + g * 32, v);
      tmem_ld_wait();
      loaded(v);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!(seen & (1u << i))) v[i] = 0xff800000u;
      tmem_st_32x32b_x32(ts + g * 32, v);
    }
    tmem_st_wait();
  }
  if (!started) {
    float top = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(ts + g * 32, v);
      tmem_ld_wait();
      loaded(v);
#pragma unroll
      for (int i = 0; i < 32; i += 2) top = max3(top, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    }
    m = top;
  }
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
    float add;
#pragma unroll 1
    while (true) {
      const float mc = m == -INFINITY ? 0.0f : (E4 ? fmaf(m, c, -kWeightLift<E4>) : m * c);
      const uint64_t cc = f32x2(c, c), mm = f32x2(-mc, -mc);
      float top[2] = {-INFINITY, -INFINITY};
      uint64_t sum[2] = {0, 0};
      uint32_t x[2][32];
      tmem_ld_32x32b_x32(ts + h * 64, x[0]);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t (&v)[32] = x[g];
        tmem_ld_wait();
        loaded(v);
        if (g == 0) tmem_ld_32x32b_x32(ts + h * 64 + 32, x[1]);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          top[0] = max3(top[0], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          top[1] = max3(top[1], __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float a, b;
          f32x2_parts(fma_f32x2(f32x2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), cc, mm), a, b);
          a = exp2_approx(a);
          b = exp2_approx(b);
          sum[q & 1] = add_f32x2(sum[q & 1], f32x2(a, b));
          // the weights as 16-bit operands (each within 2^-8 of itself in bf16; fp16: see kWeightLift)
          pk[16 * g + q] = E4 ? pack_half(a, b) : pack_bf16(a, b);
        }
      }
      float s0, s1;
      f32x2_parts(add_f32x2(sum[0], sum[1]), s0, s1);
      add = s0 + s1;
      const float mx = fmaxf(top[0], top[1]);
      const bool up = (mx - m) * c > kRaise;      // false for -inf - -inf
      if (!__any_sync(0xffffffffu, up)) break;
      const float f = up ? exp2_approx((m - mx) * c) : 1.0f;
      if (up) m = mx;
      l *= f;
      // every earlier tile's product into O is complete: these scores' commit came after them
      if (h == 1 && !half_in()) return false;
      if (started || h == 1) {
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i) {
          uint32_t o[16];
          tmem_ld_32x32b_x16(to + i * 16, o);
          tmem_ld_wait();
          loaded(o);
#pragma unroll
          for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
          tmem_st_32x32b_x16(to + i * 16, o);
        }
      }
    }
    l += add;
    tmem_st_32x32b_x32(ts + h * 32, pk);
    ready(h);
  }
  return true;
}

template <int D, bool E4>
__global__ void __launch_bounds__(TileWarps<E4>::kThreads, 1) attn_tile_kernel(const __grid_constant__ TileParams p) {
  using C = TileCfg<D, E4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* plan = reinterpret_cast<uint32_t*>(smem + C::kPlan);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);   // [stages] tile complete
  uint64_t* empty = full + C::kStages;                             // [stages] tile read
  uint64_t* raw_full = empty + C::kStages;                         // [raw stages] codes complete
  uint64_t* raw_empty = raw_full + C::kRawStages;
  uint64_t* q_full = raw_empty + C::kRawStages;                    // the piece's queries are in place
  uint64_t* q_free = q_full + 1;                                   // and have been read
  uint64_t* s_full = q_free + 1;                                   // [2] scores complete
  uint64_t* p_full = s_full + 2;                                   // [2][2] halves of the weights written
  uint64_t* h_full = p_full + 4;                                   // [2] the first half's product is in O
  uint64_t* o_full = h_full + 2;                                   // [2] output complete
  uint64_t* cleaned = o_full + 2;                                  // [stages] a value tile is cleaned
  uint64_t* drain = cleaned + C::kStages;                          // after an abort: products complete
  uint64_t* piece_full = drain + 1;                                // [pieces] told
  uint64_t* piece_empty = piece_full + kPieces;                    // [pieces] read by every role
  uint64_t* group_bar = piece_empty + kPieces;                     // [2] a softmax group meets
  uint64_t* both_bar = group_bar + 2;                              // both meet
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(both_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;                        // [2]
  volatile int* nf_item = last_flag + 2;                           // [8] pieces with non-finite hidden values
  volatile int* told = reinterpret_cast<volatile int*>(smem + C::kPieceAt);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], E4 ? 4 : 2);      // four converting warps, or the two copying ones
      mbar_init(&empty[i], E4 ? 1 : 2);     // the products, and the cleaning warp
      mbar_init(&cleaned[i], 1);
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(&raw_full[i], 2);
      mbar_init(&raw_empty[i], 4);
    }
    mbar_init(q_full, p.q_tma ? 1 : kItemRows);
    mbar_init(q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], kRowTile);
      mbar_init(&p_full[2 * i + 1], kRowTile);
      mbar_init(&h_full[i], 1);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      // 8 softmax warps, the products', the second copying one, the cleaning or converting ones
      mbar_init(&piece_empty[i], E4 ? 14 : 11);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&group_bar[i], kRowTile);
    mbar_init(both_bar, kItemRows);
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) nf_item[i] = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
    if (p.q_tma) tma_prefetch_desc(&p.tq);
  }
  // Behind the decode kernel of a call over the cache: that kernel let this one
  // start once the kernels before it had completed; its own results are not
  // read here, only its completion is waited for at the end.
  if (p.alone) pdl_wait_primary();

  // (in the shadow of the plan, whose barrier is the allocation's too)
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  tile_plan(p, plan, warp, TileWarps<E4>::kThreads / 32, lane);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_s = tmem, tm_o = tmem + 256;   // S of stream s at tm_s + 128 s, O at tm_o + D s

  uint32_t told_n = 0;
  // a bounded wait of a whole warp; false once any wait of the block ran out
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    bool ok = false;
    for (uint32_t polls = 1; !ok; ++polls) {
      ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
      if ((polls & 63u) == 0u && (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs)) break;
    }
    if (__all_sync(0xffffffffu, ok)) return true;
    if (lane == 0) {
      *abort_flag = 1;
      record_status(p.status, EPILORA_ERR_TIMEOUT);
    }
    return false;
  };
  // the next piece, as every role but the walking one gets it; false: no more
  auto next_piece = [&](Piece& q) {
    const int e = told_n % kPieces;
    if (!wait(&piece_full[e], (told_n / kPieces) & 1u)) return false;
    int* to = reinterpret_cast<int*>(&q);
#pragma unroll
    for (int i = 0; i < kPieceInts; ++i) to[i] = told[e * kPieceInts + i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[e]);
    ++told_n;
    return q.t1 > q.t0;
  };

  if (warp >= 8) {
    setmaxnreg_dec<TileWarps<E4>::kOther>();
    if (warp == 8 || warp == 11) {
      // ===== copies (of the first of the two warps: the walk and the queries too) =====
      fence_proxy_async_global();
      constexpr int kSt = E4 ? C::kRawStages : C::kStages;
      constexpr int kBytes = E4 ? C::kRawBytes : C::kTileBytes;
      constexpr int kRowBytes = E4 ? D : 128;              // inner extent of a box
      constexpr int kBoxes = E4 ? 1 : D / 64;
      uint64_t* bar_full = E4 ? raw_full : full;
      uint64_t* bar_empty = E4 ? raw_empty : empty;
      uint8_t* ring = smem + (E4 ? C::kRaw : C::kRing);
      const int nb = kPosTile / p.box_rows;                // boxes per tile along the positions
      const int part = warp == 8 ? 0 : 1;                  // copies part, part + 2, ... of a tile
      const int mine = 2 * lane + part;
      int slot = 0;
      uint32_t phase = 0, items = 0;
      TileWalk w;
      Piece it;
      bool more = part == 0 && tile_begin(p, w, plan, lane), stop = false;
      while (!stop) {
        if (part == 1) {
          if (!next_piece(it)) break;
        } else {
          // tell the piece (one that holds no tile of its item is left out)
          const int e = told_n % kPieces;
          it.t0 = it.t1 = 0;
          while (more) {
            piece_of(p, w, it);
            if (it.t1 > it.t0) break;
            more = tile_next(p, w);
          }
          if (!wait(&piece_empty[e], ((told_n / kPieces) & 1u) ^ 1u)) break;
          if (lane == 0) {
            const int* from = reinterpret_cast<const int*>(&it);
#pragma unroll
            for (int i = 0; i < kPieceInts; ++i) told[e * kPieceInts + i] = from[i];
            mbar_arrive(&piece_full[e]);
          }
          __syncwarp();
          ++told_n;
          if (!more) break;
        }
        const int32_t* table = p.paged ? p.b.page_table + it.b * p.b.table_stride : nullptr;
        auto page_of = [&](int u) {   // page of box u of the sequence
          return p.paged && u * p.box_rows < it.see_end ? table[(u * p.box_rows) >> p.page_shift] : 0;
        };
        bool q_due = !E4 && p.q_tma && part == 0;
        int c0 = it.t0 * nb;
        int ids = page_of(c0 + lane);
        for (int j = it.t0; j < it.t1 && !stop; ++j) {
          if (j * nb >= c0 + 32) {
            c0 += 32;
            ids = page_of(c0 + lane);
          }
          if (p.paged && part == 0 && (ids < 0 || ids >= p.c.num_pages))
            record_status(p.status, EPILORA_ERR_INVALID_ARG);
          const int held = min(max(it.see_end - j * kPosTile, 0), kPosTile);           // rows some row of the item sees
          const int boxes = p.paged ? (held + p.box_rows - 1) / p.box_rows : (held > 0 ? 1 : 0);
          const int copies = (boxes * kBoxes + 1 - part) / 2;                           // of this warp
          // box `mine` of the tile: rows i, columns x
          const int i = mine / kBoxes, x = mine % kBoxes;
          const int pg = __shfl_sync(0xffffffffu, ids, min(j * nb + i - c0, 31));
          const int pos = j * kPosTile + i * p.box_rows;
          // a page index out of range, and rows past the packed array, read as zeros
          const int y = p.paged ? pos & (p.c.page_size - 1) : it.first + pos;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (!wait(&bar_empty[slot], phase ^ 1u)) {
              stop = true;
              break;
            }
            uint8_t* dst = ring + slot * kBytes;
            if (lane == 0) {
              if (copies > 0)
                mbar_arrive_expect_tx(&bar_full[slot], copies * p.box_rows * kRowBytes);
              else
                mbar_arrive(&bar_full[slot]);
            }
            __syncwarp();
            if (lane < copies)
              tma_load_4d(dst + x * C::kBlock + i * p.box_rows * kRowBytes, kv ? &p.tv : &p.tk, &bar_full[slot],
                          x * kRowBytes, y, it.h, p.paged ? pg : 0);
            __syncwarp();
            if (++slot == kSt) slot = 0, phase ^= 1u;
          }
          if (!E4 && q_due && !stop) {
            // the queries, behind the first tile (by then the last piece's products are about to have read theirs)
            q_due = false;
            if (!wait(q_free, (items & 1u) ^ 1u)) {
              stop = true;
            } else if (lane == 0) {
              const int tiles = it.two() ? 2 : 1;
              mbar_arrive_expect_tx(q_full, tiles * C::kTileBytes);
              for (int t = 0; t < tiles; ++t)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  tma_load_4d(smem + t * C::kTileBytes + c * C::kBlock, &p.tq, q_full, c * 128, it.h * p.group,
                              it.first + token_of(p, it.row0 + t * kRowTile), 0);
            }
            __syncwarp();
            ++items;
          }
        }
        if (part == 0) more = tile_next(p, w);
      }
      if (*abort_flag && lane == 0) {
        // no copy in flight at exit
        for (int i = 0; i < kSt; ++i)
          (void)mbar_wait_bounded(&bar_full[i], i < slot ? phase : phase ^ 1u, 1000000ull);
        if (!E4 && p.q_tma && items > 0) (void)mbar_wait_bounded(q_full, (items - 1) & 1u, 1000000ull);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ===== products =====
      // A stream takes S = Q K^T of a tile, then (the weights having gone over
      // the scores) O += P V, then the next tile's S; the streams in turn. One
      // lane does it all, its products run in order, so no S is overwritten
      // early. A wait takes some 100 cycles even where its barrier is ready (130
      // for a whole warp), the products between two of them 256 or 512: a step's
      // barriers are therefore tried together and waited for one by one only
      // where one is not ready. (A lane per stream instead took a sixth
      // longer for a prompt of 8192 x 64 heads: the streams then fall into
      // step, and the products wait for the softmax of both.)
      if (elect_one()) {
        constexpr uint32_t kIdQK = idesc_f16(128, 128, !E4, false);
        constexpr uint32_t kIdPV = idesc_f16(128, D, !E4, true);
        const uint64_t q_desc = make_smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        const uint64_t k_desc = make_smem_desc(smem_u32(smem + C::kRing), 16, 1024, kSwizzle128B);
        const uint64_t v_desc = make_smem_desc(smem_u32(smem + C::kRing), C::kBlock, 1024, kSwizzle128B);
        constexpr uint32_t kTile16 = C::kTileBytes >> 4;
        struct Ring {
          uint32_t slot, phase;
          __device__ __forceinline__ void skip(uint32_t n) {
            slot += n;
            if (slot >= C::kStages) slot -= C::kStages, phase ^= 1u;
          }
        };
        Ring start{0, 0};                  // ring position (keys and values alternating) of the piece's first tile
        uint32_t clean_phase = 0;          // a bit per stage
        uint32_t item = 0, p_phase = 0;    // p_phase: bit s for stream s
        bool ok = true, issued = false;
        auto wait1 = [&](uint64_t* bar, uint32_t parity) {
          const uint64_t t0 = globaltimer_ns();
          for (uint32_t polls = 1;; ++polls) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((polls & 63u) == 0u && (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs)) break;
          }
          *abort_flag = 1;
          record_status(p.status, EPILORA_ERR_TIMEOUT);
          return false;
        };
        while (ok) {
          // the piece
          const int e = told_n % kPieces;
          if (!(ok = wait1(&piece_full[e], (told_n / kPieces) & 1u))) break;
          Piece it;
          int* to = reinterpret_cast<int*>(&it);
#pragma unroll
          for (int i = 0; i < kPieceInts; ++i) to[i] = told[e * kPieceInts + i];
          mbar_arrive(&piece_empty[e]);
          ++told_n;
          const int nt = it.t1 - it.t0;
          if (nt <= 0) break;
          const bool two = it.two();
          const int steps = two ? 2 * nt : nt;
          // position tile of a step: i / 2 with two row tiles, else i
          Ring kr = start, vr = start;     // keys and values of the next step's tile
          vr.skip(1);
          // scores of step i (of stream i % 2)
          auto qk = [&](int i) {
            const int s = i & 1;
            const uint64_t a = q_desc + (two && s == 1 ? kTile16 : 0), b = k_desc + kr.slot * kTile16;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k / 4) * C::kBlock + (k % 4) * 32) >> 4;
              mma_f16_ss(tm_s + s * 128, a + off, b + off, kIdQK, k > 0);
            }
            tc_commit(&s_full[s]);
            if (!(two && s == 0)) {
              tc_commit(&empty[kr.slot]);
              kr.skip(2);
            }
            if (i + 1 == steps) tc_commit(q_free);
          };
          ok = wait1(q_full, item & 1u) && wait1(&full[kr.slot], kr.phase);
          if (!ok) break;
          tc_fence_after();
          qk(0);
          issued = true;
          if (steps > 1) {
            if (!two && !(ok = wait1(&full[kr.slot], kr.phase))) break;
            tc_fence_after();
            qk(1);
          }
          static_assert(C::kStages >= 4, "the next keys are waited for before this step's values are read");
#pragma unroll 1
          for (int i = 0; i < steps; ++i) {
            const int s = i & 1, j = two ? i >> 1 : i;
            const bool more = i + 2 < steps;
            const bool new_v = !(two && s == 1), new_k = more && !(two && s == 1);
            // the value tile: cleaned first where it holds positions that some row must not see
            const bool clean = !E4 && (it.t0 + j + 1) * kPosTile > it.see_all;
            uint64_t* v_bar = clean ? &cleaned[vr.slot] : &full[vr.slot];
            const uint32_t v_par = clean ? (clean_phase >> vr.slot) & 1u : vr.phase, p_par = (p_phase >> s) & 1u;
            uint32_t rv = 1, rk = 1;
            if (new_v) rv = mbar_try_wait(v_bar, v_par);
            if (new_k) rk = mbar_try_wait(&full[kr.slot], kr.phase);
            const uint32_t rp = mbar_try_wait(&p_full[2 * s], p_par);
            if (!(rv & rk & rp)) {
              ok = (rv || wait1(v_bar, v_par)) && (rk || wait1(&full[kr.slot], kr.phase)) &&
                   (rp || wait1(&p_full[2 * s], p_par));
              if (!ok) break;
            }
            tc_fence_after();
            const uint64_t b = v_desc + vr.slot * kTile16;
            // (a stream's first product starts its sum)
#pragma unroll
            for (int k = 0; k < kPosTile / 32; ++k)
              mma_f16_ts(tm_o + s * D, tm_s + s * 128 + k * 8, b + (k * 2048 >> 4), kIdPV, i >= 2 || k > 0);
            tc_commit(&h_full[s]);
            if (!mbar_try_wait(&p_full[2 * s + 1], p_par) && !(ok = wait1(&p_full[2 * s + 1], p_par))) break;
            tc_fence_after();
#pragma unroll
            for (int k = kPosTile / 32; k < kPosTile / 16; ++k)
              mma_f16_ts(tm_o + s * D, tm_s + s * 128 + k * 8, b + (k * 2048 >> 4), kIdPV, 1u);
            p_phase ^= 1u << s;
            if (!(two && s == 0)) {
              tc_commit(&empty[vr.slot]);
              if (clean) clean_phase ^= 1u << vr.slot;
              vr.skip(2);
            }
            if (!more) tc_commit(&o_full[s]);
            if (more) {
              qk(i + 2);
            }
          }
          // 2 nt tiles further
          const uint32_t turned = start.slot + 2 * static_cast<uint32_t>(nt);
          start.slot = turned % C::kStages;
          start.phase ^= (turned / C::kStages) & 1u;
          ++item;
        }
        if (!ok && issued) {
          // no product in flight at exit: a commit covers everything issued before it
          tc_commit(drain);
          (void)mbar_wait_bounded(drain, 0, 1000000ull);
        }
      }
      __syncwarp();
    } else if (E4 ? warp >= 12 : warp == 10) {
      if (!E4) {
        // ===== cleaning of value tiles =====
        // A position that a row does not see has weight zero, but zero times a
        // NaN or an infinity is NaN: rows past the item's last position are
        // zeroed; non-finite values at positions that only some rows see are
        // zeroed too and the item noted (its epilogue adds them where they belong).
        uint32_t slot = 0, phase = 0;
        int item = 0;
        bool ok = true;
        Piece it;
        while (ok && next_piece(it)) {
          for (int j = it.t0; j < it.t1 && ok; ++j) {
            // (every fill is seen in order)
            if (!(ok = wait(&full[slot], phase))) break;
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (++slot == C::kStages) slot = 0, phase ^= 1u;
            if (!(ok = wait(&full[slot], phase))) break;
            if ((j + 1) * kPosTile > it.see_all) {
              uint8_t* v = smem + C::kRing + slot * C::kTileBytes;
              const int from = max(it.see_all - j * kPosTile, 0);
              const int to = min(max(it.see_end - j * kPosTile, from), kPosTile);
              bool nf = false;
#pragma unroll 1
              for (int x = 0; x < D / 64; ++x) {
                uint4* q = reinterpret_cast<uint4*>(v + x * C::kBlock);
                for (int i = to * 8 + lane; i < kPosTile * 8; i += 32) q[i] = make_uint4(0, 0, 0, 0);
                for (int i0 = from * 8 + lane; i0 < to * 8; i0 += 128) {
                  uint4 u[4];
                  bool any = false;
#pragma unroll
                  for (int k = 0; k < 4; ++k) u[k] = i0 + 32 * k < to * 8 ? q[i0 + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    any |= bf16x2_nonfinite(u[k].x) | bf16x2_nonfinite(u[k].y) | bf16x2_nonfinite(u[k].z) |
                           bf16x2_nonfinite(u[k].w);
                  if (any) {
                    nf = true;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      uint32_t e[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                      for (int y = 0; y < 4; ++y) {
                        if ((e[y] & 0x7F80u) == 0x7F80u) e[y] &= 0xFFFF0000u;
                        if ((e[y] & 0x7F800000u) == 0x7F800000u) e[y] &= 0xFFFFu;
                      }
                      if (i0 + 32 * k < to * 8) q[i0 + 32 * k] = make_uint4(e[0], e[1], e[2], e[3]);
                    }
                  }
                }
              }
              if (nf) nf_item[item & 7] = item + 1;
              fence_proxy_async_smem();
              __threadfence_block();
              __syncwarp();
              if (lane == 0) mbar_arrive(&cleaned[slot]);
            }
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (++slot == C::kStages) slot = 0, phase ^= 1u;
          }
          ++item;
        }
      } else {
        // ===== E4M3 codes to fp16 tiles =====
        const int t = (warp - 12) * 32 + lane;
        uint32_t slot = 0, phase = 0, rslot = 0, rphase = 0;
        int item = 0;
        bool ok = true;
        Piece it;
        while (ok && next_piece(it)) {
          for (int j = it.t0; j < it.t1 && ok; ++j) {
            const int from = max(it.see_all - j * kPosTile, 0);
            const int to = min(max(it.see_end - j * kPosTile, 0), kPosTile);
            for (int kv = 0; kv < 2 && ok; ++kv) {
              ok = wait(&raw_full[rslot], rphase) && wait(&empty[slot], phase ^ 1u);
              if (!ok) break;
              const uint8_t* src = smem + C::kRaw + rslot * C::kRawBytes;
              uint8_t* dst = smem + C::kRing + slot * C::kTileBytes;
              bool nf = false;
              const bool clean = kv == 1 && from < kPosTile;
              // A thread takes 16-code chunk c of the rows r0, r0 + kStep, ...: chunks
              // 2c and 2c + 1 of the 16-bit row's 16-byte chunks, swizzled alike in
              // all of its rows (kStep is a multiple of 8). The two halves of a
              // 128-element row store theirs in opposite order, so that they use
              // different banks.
              constexpr int kPer = D / 16, kStep = 128 / kPer;
              const int r0 = t / kPer, c = t % kPer, first = (c / 4) & 1;
              uint8_t* row_at = dst + (c / 4) * C::kBlock + r0 * 128;
              const uint32_t at0 = (((c % 4) * 2 + first) ^ (r0 & 7)) * 16, at1 = at0 ^ 16u;
              auto store = [&](int y, const uint4& u) {
                uint4 lo, hi;
                lo.x = e4m3x2_to_f16x2(u.x), lo.y = e4m3x2_to_f16x2(u.x >> 16);
                lo.z = e4m3x2_to_f16x2(u.y), lo.w = e4m3x2_to_f16x2(u.y >> 16);
                hi.x = e4m3x2_to_f16x2(u.z), hi.y = e4m3x2_to_f16x2(u.z >> 16);
                hi.z = e4m3x2_to_f16x2(u.w), hi.w = e4m3x2_to_f16x2(u.w >> 16);
                *reinterpret_cast<uint4*>(row_at + at0 + y * kStep * 128) = first ? hi : lo;
                *reinterpret_cast<uint4*>(row_at + at1 + y * kStep * 128) = first ? lo : hi;
              };
              const uint4* codes = reinterpret_cast<const uint4*>(src) + t;
              if (!clean) {
                // (no branch in the body: its loads and conversions overlap)
#pragma unroll 1
                for (int y = 0; y < kPer; y += 4) {
                  uint4 u[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) u[k] = codes[(y + k) * 128];
#pragma unroll
                  for (int k = 0; k < 4; ++k) store(y + k, u[k]);
                }
              } else {
#pragma unroll 1
                for (int y = 0; y < kPer; ++y) {
                  uint4 u = codes[y * 128];
                  const int row = r0 + y * kStep;
                  if (row >= to) {
                    u = make_uint4(0, 0, 0, 0);
                  } else if (row >= from && (e4m3x4_nan(u.x) | e4m3x4_nan(u.y) | e4m3x4_nan(u.z) | e4m3x4_nan(u.w))) {
                    nf = true;
                    u.x = e4m3x4_strip_nan(u.x), u.y = e4m3x4_strip_nan(u.y);
                    u.z = e4m3x4_strip_nan(u.z), u.w = e4m3x4_strip_nan(u.w);
                  }
                  store(y, u);
                }
              }
              if (nf) nf_item[item & 7] = item + 1;
              fence_proxy_async_smem();
              __threadfence_block();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&full[slot]);
                mbar_arrive(&raw_empty[rslot]);
              }
              if (++slot == C::kStages) slot = 0, phase ^= 1u;
              if (++rslot == C::kRawStages) rslot = 0, rphase ^= 1u;
            }
          }
          ++item;
        }
      }
    }
  } else {
    // ===== softmax =====
    setmaxnreg_inc<TileWarps<E4>::kSoftmax>();
    if (p.alone) {
      // packed rows of no sequence are zero (the decode kernel's part where there is one); here, before the first
      // scores are there, it costs nothing
      const int used = p.b.n_seqs > 0 ? min(max(p.b.q_start[p.b.n_seqs], 0), p.b.n_tokens) : 0;
      const int64_t rows = static_cast<int64_t>(p.b.n_tokens - used) * p.heads;
      constexpr int V = D / 8;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * kItemRows + threadIdx.x; i < rows * V;
           i += static_cast<int64_t>(gridDim.x) * kItemRows) {
        const int64_t r = i / V;
        const int64_t t = used + r / p.heads;
        const int h = static_cast<int>(r % p.heads);
        *reinterpret_cast<uint4*>(p.o.p + t * p.o.ts + h * p.o.hs + (i % V) * 8) = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr && i % V == 0) p.lse[t * p.heads + h] = -INFINITY;
      }
    }
    const int s = warp >> 2;                       // stream
    const int r = threadIdx.x & (kRowTile - 1);    // lane of TMEM = row of the stream
    const uint32_t quad = static_cast<uint32_t>(warp & 3) << 21;   // TMEM lane 32 (warp % 4), in bits 16..
    const uint32_t ts = tm_s + s * 128 + quad, to = tm_o + s * D + quad;
    uint32_t sn = 0, on[2] = {0, 0};
    int item = 0;
    uint32_t group_n = 0, both_n = 0;
    auto meet_group = [&]() {
      mbar_arrive(&group_bar[s]);
      return wait(&group_bar[s], group_n++ & 1u);
    };
    auto meet_both = [&]() {
      mbar_arrive(both_bar);
      return wait(both_bar, both_n++ & 1u);
    };
    float* other = reinterpret_cast<float*>(smem + C::kPlan);   // m, l of stream 1 (the plan has been read)
    Piece it;
    // a wait that ran out ends the loop at once: no barrier in it waits for ever
    while (next_piece(it)) {
      const int nt = it.t1 - it.t0;
      const bool two = it.two();
      const int lrow = two ? s * kRowTile + r : r;      // row within the item
      const bool live = lrow < it.rows;
      const int grow = it.row0 + (live ? lrow : 0);
      const int new_tok = token_of(p, grow);
      const int64_t tok = it.first + new_tok;
      const int head = it.h * p.group + grow - new_tok * p.group;
      const int see = live ? max(min(it.base + new_tok + 1, it.len), 0) : 0;
      float s_eff = p.scale;
      if (E4) s_eff *= p.c.k_scale[it.h];
      float c = s_eff == 0.0f ? 1.0f : fabsf(s_eff) * kLog2e;

      // the row of queries into shared memory (swizzled, K-major), where no copy does it
      if (E4 || !p.q_tma) {
        const __nv_bfloat16* src = p.q.p + tok * p.q.ts + head * p.q.hs;
        const bool use = live && s_eff != 0.0f;
        const uint32_t flip = s_eff < 0.0f ? 0x80008000u : 0u;
        uint4 u[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          u[i] = use ? *reinterpret_cast<const uint4*>(src + i * 8) : make_uint4(0, 0, 0, 0);
        if (E4) {
          // fp16 queries: bf16's 8 significant bits fit; the row is scaled by
          // the power of two that puts its largest element near 2^13
          // (elements 2^27 below that are still exact, the rest is off by
          // 2^-38 of the largest), the scores' factor takes it back
          float big = 0.0f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint32_t e[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(bf16_lo(e[k])), fabsf(bf16_hi(e[k]))));
          }
          const int ex = static_cast<int>((__float_as_uint(big) >> 23) & 0xFF);
          const int up = big == 0.0f || ex == 0xFF ? 0 : min(13 - (ex - 127), 126);
          const float f = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
          if (up != 0) c *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            u[i].x = pack_half(bf16_lo(u[i].x) * f, bf16_hi(u[i].x) * f);
            u[i].y = pack_half(bf16_lo(u[i].y) * f, bf16_hi(u[i].y) * f);
            u[i].z = pack_half(bf16_lo(u[i].z) * f, bf16_hi(u[i].z) * f);
            u[i].w = pack_half(bf16_lo(u[i].w) * f, bf16_hi(u[i].w) * f);
          }
        }
        if (two || s == 0) {
          uint8_t* dst = smem + s * C::kTileBytes + r * 128;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = make_uint4(u[i].x ^ flip, u[i].y ^ flip, u[i].z ^ flip, u[i].w ^ flip);
            *reinterpret_cast<uint4*>(dst + (i / 8) * C::kBlock + (((i & 7) ^ (r & 7)) * 16)) = v;
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(q_full);
      }

      float m = -INFINITY, l = 0.0f;   // m in units of S
      const int steps = two ? nt : (nt + 1 - s) / 2;
      int lim = see - (it.t0 + (two ? 0 : s)) * kPosTile;     // the row sees the tile's columns below lim
      const int lim_step = two ? kPosTile : 2 * kPosTile;
      bool started = false;
#pragma unroll 1
      for (int k = 0; k < steps; ++k) {
        if (!wait(&s_full[s], sn++ & 1u)) break;
        tc_fence_after();
        const bool done = softmax_tile<D, E4>(
            ts, to, c, lim, started, m, l,
            [&](int half) {
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(&p_full[2 * s + half]);
            },
            [&]() {
              if (!wait(&h_full[s], (sn - 1) & 1u)) return false;
              tc_fence_after();
              return true;
            });
        if (!done) break;
        started = true;
        lim -= lim_step;
      }

      // ===== the piece's result =====
      if (steps > 0 && !wait(&o_full[s], on[s]++ & 1u)) break;
      float f0 = 1.0f, f1 = 0.0f;      // factors of the two streams' outputs
      bool both = false;
      if (!two) {
        if (s == 1) other[r] = m, other[kRowTile + r] = l;
        if (!meet_both()) break;
        if (s == 0) {
          both = nt > 1;
          if (both) {
            if (!wait(&o_full[1], on[1]++ & 1u)) break;
            const float m1 = other[r], l1 = other[kRowTile + r];
            const float mm = fmaxf(m, m1);
            const float base = mm == -INFINITY ? 0.0f : mm;
            f0 = exp2_approx((m - base) * c);
            f1 = exp2_approx((m1 - base) * c);
            l = l * f0 + l1 * f1;
            m = mm;
          }
        }
      } else if (s == 0) {
        ++on[1];     // keep count of the other stream's outputs
      }
      tc_fence_after();
      if (two || s == 0) {
        const bool whole = it.whole != 0;
        const float vscale = E4 ? p.c.v_scale[it.h] : 1.0f;
        const bool nf = nf_item[item & 7] == item + 1;
        constexpr int kPart = (2 + D) * kItemRows / 4;      // float4s of a partial result: m c, l, O [D / 4][256]
        float4* part = p.partials + static_cast<int64_t>(it.slot) * kPart;
        const int prow = s * kRowTile + r;
        auto put = [&](int i, const float* o, float inv, bool empty) {   // 32 outputs from element i on
          uint32_t v[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = empty ? 0u : pack_bf16(o[2 * q] * inv, o[2 * q + 1] * inv);
          __nv_bfloat16* at = p.o.p + tok * p.o.ts + head * p.o.hs + i;
          if (p.o_sectors) {
            st_global_v8(at, v);
            st_global_v8(at + 16, v + 8);
          } else {
#pragma unroll
            for (int q = 0; q < 16; q += 4)
              *reinterpret_cast<uint4*>(at + 2 * q) = make_uint4(v[q], v[q + 1], v[q + 2], v[q + 3]);
          }
        };
        auto put_lse = [&](float mc, float sum) {
          if (p.lse != nullptr) p.lse[tok * p.heads + head] = sum == 0.0f ? -INFINITY : (mc + __log2f(sum)) * kLn2;
        };
        const float inv = vscale / l;      // (l == 0: the row sees nothing)
        const bool plain = whole && !both && p.o_sectors;
        if (plain) {
          // the usual case: the next 32 columns on their way while these are stored
          __nv_bfloat16* at = p.o.p + tok * p.o.ts + head * p.o.hs;
          const uint64_t inv2 = f32x2(inv, inv);
          const bool empty = l == 0.0f;
          uint32_t o[2][32];
          tmem_ld_32x32b_x32(to, o[0]);
#pragma unroll 1
          for (int i0 = 0; i0 < D; i0 += 64) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t (&x)[32] = o[y];
              const int i = i0 + 32 * y;
              tmem_ld_wait();
              loaded(x);
              if (i + 32 < D) tmem_ld_32x32b_x32(to + i + 32, o[y ^ 1]);
              uint32_t v[16];
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                float a, b;
                f32x2_parts(mul_f32x2(f32x2(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1])), inv2), a, b);
                v[q] = empty ? 0u : pack_bf16(a, b);
              }
              if (live) {
                st_global_v8(at + i, v);
                st_global_v8(at + i + 16, v + 8);
              }
            }
          }
        }
#pragma unroll 1
        for (int i = 0; i < D && !plain; i += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tm_o + s * D + quad + i, o);
          tmem_ld_wait();
          loaded(o);
          float a[32];
#pragma unroll
          for (int q = 0; q < 32; ++q) a[q] = __uint_as_float(o[q]);
          if (!two && both) {
            tmem_ld_32x32b_x32(tm_o + D + quad + i, o);
            tmem_ld_wait();
            loaded(o);
#pragma unroll
            for (int q = 0; q < 32; ++q) a[q] = a[q] * f0 + __uint_as_float(o[q]) * f1;
          }
          if (whole) {
            if (live) {
              put(i, a, inv, l == 0.0f);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 32; q += 4)
              part[2 * kItemRows / 4 + (i + q) / 4 * kItemRows + prow] =
                  make_float4(a[q], a[q + 1], a[q + 2], a[q + 3]);
          }
        }
        // as in softmax_tile: the maximum less the lift
        const float mc = m == -INFINITY ? -INFINITY : (E4 ? fmaf(m, c, -kWeightLift<E4>) : m * c);
        if (nf) {
          // the non-finite values that were taken out, where this row sees them, go into what was just written
          const int to_pos = live ? min(see, it.t1 * kPosTile) : 0;
#pragma unroll 1
          for (int pos = max(it.see_all, it.t0 * kPosTile); pos < to_pos; ++pos) {
            const __nv_bfloat16* v = nullptr;
            const uint8_t* v4 = nullptr;
            if (!p.paged) {
              v = p.v.p + (it.first + pos) * p.v.ts + it.h * p.v.hs;
            } else {
              const int pg = p.b.page_table[it.b * p.b.table_stride + (pos >> p.page_shift)];
              if (pg < 0 || pg >= p.c.num_pages) continue;
              const int64_t at = pg * p.c.v_page_stride + it.h * p.c.v_head_stride +
                                 (pos & (p.c.page_size - 1)) * p.c.v_token_stride;
              v = static_cast<const __nv_bfloat16*>(p.c.v) + at;
              v4 = static_cast<const uint8_t*>(p.c.v) + at;
            }
#pragma unroll 1
            for (int i = 0; i < D; ++i) {
              const float e = E4 ? e4m3_to_f32(v4[i]) : __bfloat162float(v[i]);
              if (fabsf(e) < INFINITY) continue;
              if (whole) {
                __nv_bfloat16* o = p.o.p + tok * p.o.ts + head * p.o.hs + i;
                *o = __float2bfloat16_rn(__bfloat162float(*o) + e);
              } else {
                float* o = reinterpret_cast<float*>(part + 2 * kItemRows / 4 + i / 4 * kItemRows + prow) + i % 4;
                *o += e;
              }
            }
          }
        }
        if (whole) {
          if (live) put_lse(mc, l);
        } else {
          float* pf = reinterpret_cast<float*>(part);
          pf[prow] = mc;
          pf[kItemRows + prow] = l;
          const int first = it.first_cta, pieces = it.pieces;
          if (!meet_group()) break;
          if (r == 0) {
            // (the group's stores are before it: the barrier above)
            const int is_last = atom_inc_acq_rel_gpu(p.counters + 2 * first + s) == static_cast<uint32_t>(pieces - 1);
            if (is_last) p.counters[2 * first + s] = 0;
            last_flag[s] = is_last;
          }
          if (!meet_group()) break;
          if (last_flag[s] && live) {
            auto piece = [&](int k) {
              return p.partials + static_cast<int64_t>(k == 0 ? it.slot0 : 2 * (first + k)) * kPart;
            };
            float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
            for (int k = 0; k < pieces; ++k) {
              const float* f = reinterpret_cast<const float*>(piece(k));
              const float mk = __ldcg(f + prow), lk = __ldcg(f + kItemRows + prow);
              const float up = fmaxf(top, mk), to = up == -INFINITY ? 0.0f : up;
              sum = sum * exp2_approx(top - to) + lk * exp2_approx(mk - to);
              top = up;
            }
            const float base = top == -INFINITY ? 0.0f : top;
            const float inv = vscale / sum;
            // 64 columns of a piece at a time: the loads are what a join waits for (four prompts of 37 new tokens,
            // cut into ten pieces each: 32.0 us with 32 columns at a time, 29.4 so)
#pragma unroll 1
            for (int i = 0; i < D; i += 64) {
              float a[64];
#pragma unroll
              for (int q = 0; q < 64; ++q) a[q] = 0.0f;
#pragma unroll 1
              for (int k = 0; k < pieces; ++k) {
                const float4* f = piece(k);
                const float mk = __ldcg(reinterpret_cast<const float*>(f) + prow);
                float4 x[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) x[q] = __ldcg(f + 2 * kItemRows / 4 + (i / 4 + q) * kItemRows + prow);
                const float wk = exp2_approx(mk - base);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                  a[4 * q] += x[q].x * wk, a[4 * q + 1] += x[q].y * wk;
                  a[4 * q + 2] += x[q].z * wk, a[4 * q + 3] += x[q].w * wk;
                }
              }
              put(i, a, inv, sum == 0.0f);
              put(i + 32, a + 32, inv, sum == 0.0f);
            }
            put_lse(top, sum);
          }
        }
        tc_fence_before();
      }
      if (!two && !meet_both()) break;    // both streams' outputs and `other` are free again
      ++item;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (!p.alone) pdl_wait_primary();
}

// Whether a tile's 128 rows are a box [tokens][group heads] of the queries, to
// be used as they are: the group divides the tile, the scale needs no change of
// sign. (Other queries are loaded by the softmax threads, which then start a
// piece only when the last one's output is written: 3.5 us later.)
bool q_boxes_fit(const TileParams& p, const AttnArgs& a) { return kRowTile % p.group == 0 && a.scale > 0.0f; }

template <int D, bool E4>
int launch(const AttnArgs& a, TileParams& p) {
  using C = TileCfg<D, E4>;
  const uint64_t es = E4 ? 1 : 2;
  const uint32_t inner = E4 ? D : 128;
  int rc;
  if (a.paged) {
    const epilora_kv_cache& c = a.cache;
    const uint64_t dims[4] = {D * es, static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(c.kv_heads),
                              static_cast<uint64_t>(c.num_pages)};
    const uint32_t box[4] = {inner, static_cast<uint32_t>(p.box_rows), 1, 1};
    const uint64_t ks[3] = {c.k_token_stride * es, c.k_head_stride * es, c.k_page_stride * es};
    const uint64_t vs[3] = {c.v_token_stride * es, c.v_head_stride * es, c.v_page_stride * es};
    rc = make_tma_4d_u8(&p.tk, c.k, dims, ks, box, E4 ? 0 : 128);
    if (rc == EPILORA_OK) rc = make_tma_4d_u8(&p.tv, c.v, dims, vs, box, E4 ? 0 : 128);
  } else {
    const uint64_t T = static_cast<uint64_t>(a.batch.n_tokens);
    const uint64_t dims[4] = {D * es, T, static_cast<uint64_t>(a.cache.kv_heads), 1};
    const uint32_t box[4] = {inner, kPosTile, 1, 1};
    const uint64_t ks[3] = {a.k.ts * es, a.k.hs * es, a.k.ts * es * T};
    const uint64_t vs[3] = {a.v.ts * es, a.v.hs * es, a.v.ts * es * T};
    rc = make_tma_4d_u8(&p.tk, a.k.p, dims, ks, box, 128);
    if (rc == EPILORA_OK) rc = make_tma_4d_u8(&p.tv, a.v.p, dims, vs, box, 128);
  }
  if (rc == EPILORA_OK && !E4 && q_boxes_fit(p, a)) {
    const uint64_t T = static_cast<uint64_t>(a.batch.n_tokens);
    const uint64_t dims[4] = {D * 2, static_cast<uint64_t>(a.heads), T, 1};
    const uint32_t box[4] = {128, static_cast<uint32_t>(p.group), static_cast<uint32_t>(kRowTile / p.group), 1};
    const uint64_t hs = a.q.hs * es, ts = a.q.ts * es;
    const uint64_t qs[3] = {hs, ts, ts * T};
    rc = make_tma_4d_u8(&p.tq, a.q.p, dims, qs, box, 128);
    p.q_tma = 1;
  }
  if (rc != EPILORA_OK) return rc;
  auto kern = attn_tile_kernel<D, E4>;
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EPILORA_ERR_CUDA;
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return EPILORA_ERR_CUDA;
    attr_done[dev] = 1;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(num_sms() < kTileMaxCtas ? num_sms() : kTileMaxCtas, 1, 1);
  cfg.blockDim = dim3(TileWarps<E4>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

}  // namespace

size_t attn_tile_counter_bytes() { return 2 * kTileMaxCtas * sizeof(uint32_t); }
size_t attn_tile_partial_bytes(int head_dim) {
  const int n = num_sms() < kTileMaxCtas ? num_sms() : kTileMaxCtas;
  return static_cast<size_t>(2 * n) * (2 + head_dim) * kItemRows * sizeof(float);
}

bool attn_tile_fits(const AttnArgs& a) {
  const double longest =
      a.paged ? static_cast<double>(a.batch.table_pages) * a.cache.page_size : static_cast<double>(a.batch.n_tokens);
  const double items = static_cast<double>(a.batch.n_tokens) * a.heads / kItemRows +
                       static_cast<double>(a.batch.n_seqs) * a.cache.kv_heads;
  return items * (longest / kPosTile + 1 + kItemCost) < 4e9;
}

int launch_attn_tile(const AttnArgs& a, bool alone, uint32_t* counters, float* partials) {
  TileParams p{};
  p.b = a.batch;
  p.c = a.cache;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.o = a.o;
  p.lse = a.lse;
  p.paged = a.paged;
  p.alone = alone;
  p.heads = a.heads;
  p.kv_heads = a.cache.kv_heads;
  p.group = a.heads / a.cache.kv_heads;
  int s = 0;
  while ((1 << s) < p.group) ++s;
  p.group_shift = 31 + s;
  p.group_mul = static_cast<uint32_t>(((uint64_t{1} << p.group_shift) + p.group - 1) / p.group);
  p.page_shift = a.paged ? __builtin_ctz(a.cache.page_size) : 0;
  p.box_rows = a.paged && a.cache.page_size < kPosTile ? a.cache.page_size : kPosTile;
  p.o_sectors = (reinterpret_cast<uintptr_t>(a.o.p) | static_cast<uintptr_t>(a.o.ts * 2) |
                 static_cast<uintptr_t>(a.o.hs * 2)) % 32 == 0;
  p.scale = a.scale;
  p.counters = counters;
  p.partials = reinterpret_cast<float4*>(partials);
  p.status = a.status;
  const bool e4 = a.paged && a.cache.kv_fmt == EPILORA_KV_E4M3;
  if (a.cache.head_dim == 64) return e4 ? launch<64, true>(a, p) : launch<64, false>(a, p);
  return e4 ? launch<128, true>(a, p) : launch<128, false>(a, p);
}

}  // namespace epi
