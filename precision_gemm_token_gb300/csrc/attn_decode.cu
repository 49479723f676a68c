// Attention of a few new tokens over the paged cache: sequences whose new
// tokens times the heads of a key/value group are at most 16 rows (one decode
// token with up to 16 heads a group, a few drafted tokens).
//
//   O = sum_j exp2(x_j - m) V_j / sum_j exp2(x_j - m),  x = (scale log2 e) q . K_j
//
// One pass over the cache with a running maximum m and sum per row. It is
// bound by reading the cache once: 2 head_dim elements per position and
// key/value head against 4 head_dim flops per query row, so the 16-row tensor
// core tile (mma.sync m16n8k16, rows = the group's heads) costs nothing even
// where 4 or 8 of its rows are used.
//
// The cache's positions are cut into tiles; the tiles of all (sequence, head)
// pairs form one line that is split evenly over the thread blocks (two per
// SM), so that any mix of lengths loads every SM alike; a pair cut between
// blocks is joined by the block that finishes last, in the order of the pieces
// (results do not depend on which block that is).
// A block is four computing warps, a copying and a joining one. The copying
// warp brings 32 positions a slot (keys and values) into a ring by TMA, in
// boxes of up to 32 rows of a page, so every layout with contiguous heads costs
// the same (with 16 positions a slot its 700 cycles a slot were the bound). A
// computing warp takes its positions of a tile with a maximum, sum and output
// of its own, so no barrier stands in its loop: 16 positions of bf16, which
// leaves it waiting for memory; 32 of E4M3, whose half as many bytes leave
// half the time, for the chains of products of two 16s side by side. At the
// end of a pair it hands its result to the joining warp and goes on: writing a
// piece's result out and learning whether it was the last takes 5 us while the
// memory is busy, and as long again to join.
//
// Measured (heads of 128): 64 sequences of up to 16384, 64 / 8 heads, 335 us
// (6.9 TB/s) in bf16, 214 us (5.4 TB/s) in E4M3, where the chains of products in
// eight computing warps an SM are the bound; 32 of up to 4096, 32 / 8 heads,
// 52.4 us (5.2 TB/s); one of 1023, 10.0 us.
#include "attention.cuh"
#include "ptx.cuh"

namespace epi {
namespace {

constexpr int kDecGroup = 32;        // positions per ring slot
constexpr int kDecWarps = 4;         // computing warps
constexpr int kDecThreads = 32 * (kDecWarps + 2);
constexpr int kDecRows = 16;
constexpr int kDecMaxCtas = 512;     // blocks of a launch at most
constexpr int kDecPieces = 4;        // pieces of work told ahead
constexpr int kDecJoin = 16;         // pieces of a join whose factors are kept
constexpr int kDecPieceInts = 12;
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

template <int D, bool E4>
struct DecCfg {
  static constexpr int kUnit = E4 ? 32 : 16;                            // positions per warp and tile
  static constexpr int kTile = kUnit * kDecWarps;                       // positions per tile
  static constexpr int kPerSlot = kDecGroup / kUnit;                    // warps that share a slot
  static constexpr int kSlotStep = kDecWarps / kPerSlot;                // slots per tile
  static constexpr int kRowBytes = D * (E4 ? 1 : 2);
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;   // inner extent = swizzle span
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  static constexpr int kUnitBytes = kUnit * kBoxBytes;                  // a warp's rows of a box column
  static constexpr int kBox = kDecGroup * kBoxBytes;                    // bytes of a box column of a slot
  static constexpr int kHalf = kBoxes * kBox;                           // keys, then values
  static constexpr int kSlotBytes = 2 * kHalf;
  // a slot always belongs to the same warps, which wait for its fills in order
  // (a warp ahead of a slot's other readers would take the parity of the fill
  // before last for its own)
  static constexpr int kSlots = 64 * 1024 / kSlotBytes;
  static_assert(kSlots % kSlotStep == 0, "slots are dealt to the warps");
  static constexpr int kOld = D + 8;                                    // floats per row of the meeting buffer
  static constexpr int kMeet = kDecWarps * kDecRows * kOld * 4;         // the four warps' outputs
  static constexpr int kSmem = 1024 + kSlots * kSlotBytes + kMeet + 3 * 1024;
};

struct DecParams {
  CUtensorMap tk, tv;
  epilora_kv_batch b;
  AttnRows q;
  AttnOut o;
  float* lse;
  int heads, kv_heads, group;
  int page_shift, page_size, num_pages;
  int box_rows;         // rows per TMA box
  float scale;
  const float* k_scale;
  const float* v_scale;
  uint32_t* counters;   // [gridDim.x], zero between calls
  float* partials;      // [2 gridDim.x][32 + 16 D]
  int* status;
};

// A sequence of this kernel's class.
struct DecSeq {
  int first, n, len, base;   // packed rows, tokens in the cache (clamped), position of new token 0
  int tiles;                 // 0: not of this class
};
template <int TILE>
__device__ __forceinline__ DecSeq dec_seq(const DecParams& p, int b, bool& bad) {
  DecSeq s;
  const SeqRows r = seq_rows(p.b.q_start, b, p.b.n_tokens, bad);
  const int len = p.b.kv_len[b];
  const int cap = p.b.table_pages << p.page_shift;
  if (len > cap || len < 0 || r.n > p.b.max_new) bad = true;
  s.first = r.first;
  s.n = r.n;
  s.base = len - r.n;
  s.len = max(min(len, cap), 0);
  s.tiles = r.n > 0 && attn_decode_takes(r.n, p.group) ? max((s.len + TILE - 1) / TILE, 1) : 0;
  return s;
}

// Walks the pieces of a thread block's range of the line of tiles (one warp).
struct DecWalk {
  uint32_t x, end;     // tiles still to do: [x, end)
  uint32_t each, more; // tiles per block: each + 1 for the first `more` blocks, else each
  int b, h;
  DecSeq s;
  int t0, t1;          // this piece's tiles of the pair
  uint32_t pair0;      // line position of the pair's tile 0
  __device__ __forceinline__ uint32_t start_of(uint32_t cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ uint32_t owner_of(uint32_t tile) const {
    const uint32_t low = more * (each + 1);
    return tile < low ? tile / (each + 1) : more + (tile - low) / each;
  }
};

__device__ __forceinline__ uint32_t dec_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__device__ __forceinline__ void dec_piece(DecWalk& w) {
  w.t0 = static_cast<int>(w.x - w.pair0);
  w.t1 = static_cast<int>(min(static_cast<uint32_t>(w.s.tiles - w.t0), w.end - w.x)) + w.t0;
}

// One warp; false: nothing to do.
template <int TILE>
__device__ __forceinline__ bool dec_begin(const DecParams& p, DecWalk& w, int lane) {
  // tiles of the sequences lane, lane + 32, ...; up to 128 sequences are read once
  constexpr int kKept = 4;
  uint32_t kept[kKept], sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int b = lane + 32 * i;
    kept[i] = b < p.b.n_seqs ? dec_seq<TILE>(p, b, bad).tiles : 0;
    sum += kept[i];
  }
  for (int b = lane + 32 * kKept; b < p.b.n_seqs; b += 32) sum += dec_seq<TILE>(p, b, bad).tiles;
  if (bad && blockIdx.x == 0) record_status(p.status, EPILORA_ERR_INVALID_ARG);
  const uint32_t total = __reduce_add_sync(0xffffffffu, sum) * p.kv_heads;
  // two tiles a block at least: a pair then has half as many pieces to join
  // (1023 positions, 8 heads: 11.7 us with one)
  const uint32_t ctas = min(gridDim.x, (total + 1) / 2);
  if (blockIdx.x >= ctas) return false;
  w.each = total / ctas;
  w.more = total - w.each * ctas;
  w.x = w.start_of(blockIdx.x);
  w.end = w.start_of(blockIdx.x + 1);
  // the sequence that holds x
  uint32_t before = 0;
  for (int i = 0;; ++i) {
    if (32 * i >= p.b.n_seqs) return false;   // metadata changed under the call
    const int b = lane + 32 * i;
    const uint32_t tiles = i < kKept ? (i == 0 ? kept[0] : i == 1 ? kept[1] : i == 2 ? kept[2] : kept[3])
                                     : (b < p.b.n_seqs ? dec_seq<TILE>(p, b, bad).tiles : 0);
    const uint32_t c = tiles * p.kv_heads, inc = dec_scan(c, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > w.x);
    if (hit != 0) {
      const int l = __ffs(hit) - 1;
      w.b = 32 * i + l;
      w.pair0 = before + __shfl_sync(0xffffffffu, inc - c, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  w.s = dec_seq<TILE>(p, w.b, bad);
  w.h = static_cast<int>((w.x - w.pair0) / w.s.tiles);
  w.pair0 += static_cast<uint32_t>(w.h) * w.s.tiles;
  dec_piece(w);
  return true;
}

template <int TILE>
__device__ __forceinline__ bool dec_next(const DecParams& p, DecWalk& w) {
  w.x += w.t1 - w.t0;
  if (w.x >= w.end) return false;
  w.pair0 += w.s.tiles;
  if (++w.h == p.kv_heads) {
    w.h = 0;
    bool bad = false;
    do {   // x < end: a sequence of the class follows
      if (++w.b >= p.b.n_seqs) return false;
      w.s = dec_seq<TILE>(p, w.b, bad);
    } while (w.s.tiles == 0);
  }
  dec_piece(w);
  return true;
}

// A piece as the walking warp tells it to the others.
struct DecPiece {
  int first, n, len, base;   // as in DecSeq
  int h;
  int t0, t1;                // tiles; t0 == t1: no more work
  int whole;                 // the pair's only piece
  int first_cta, pieces;     // of a pair in several pieces: the blocks first_cta, ...
  int slot, slot0;           // where this piece's, and the first piece's, partial result goes
};
static_assert(sizeof(DecPiece) == 4 * kDecPieceInts, "one int per field");

__device__ __forceinline__ DecPiece dec_piece_of(const DecWalk& w) {
  DecPiece q;
  q.first = w.s.first, q.n = w.s.n, q.len = w.s.len, q.base = w.s.base;
  q.h = w.h;
  q.t0 = w.t0, q.t1 = w.t1;
  q.whole = w.t0 == 0 && w.t1 == w.s.tiles;
  // the blocks that hold the pair's first and last tile
  q.first_cta = static_cast<int>(w.owner_of(w.pair0));
  q.pieces = static_cast<int>(w.owner_of(w.pair0 + w.s.tiles - 1)) - q.first_cta + 1;
  // a piece that starts its block's range goes to the block's slot 0, the one that ends it to slot 1
  q.slot = 2 * blockIdx.x + (w.x == w.start_of(blockIdx.x) ? 0 : 1);
  q.slot0 = 2 * q.first_cta + (w.start_of(q.first_cta) == w.pair0 ? 0 : 1);
  return q;
}

template <bool E4>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (E4)
    mma_f16_m16n8k16(d, a, b0, b1);
  else
    mma_bf16_m16n8k16(d, a, b0, b1);
}

template <bool E4>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (E4) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// shared-memory byte of (row, byte) in a box with rows of SPAN bytes, swizzled
// over the span by the TMA copy
template <int SPAN>
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t byte) {
  const uint32_t a = row * SPAN + byte;
  return a ^ (((a >> 7) & (SPAN / 16 - 1)) << 4);
}

// O += P V over 16 positions. SEL: only the rows of one token take the result
// (sel0 / sel1: the thread's rows g and g + 8).
template <int D, bool E4, bool SEL>
__device__ __forceinline__ void dec_pv(float (&acc)[D / 8][4], const uint32_t (&pa)[4], const uint8_t* vs, int lane,
                                       bool sel0, bool sel1) {
  using C = DecCfg<D, E4>;
  const int g = lane >> 2, q = lane & 3;
  auto add = [&](int nt, uint32_t b0, uint32_t b1) {
    if (SEL) {
      float t[4] = {acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]};
      mma16<E4>(t, pa, b0, b1);
      if (sel0) acc[nt][0] = t[0], acc[nt][1] = t[1];
      if (sel1) acc[nt][2] = t[2], acc[nt][3] = t[3];
    } else {
      mma16<E4>(acc[nt], pa, b0, b1);
    }
  };
  if (!E4) {
    const uint32_t base = smem_u32(vs);
    const uint32_t tok = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int np = 0; np < D / 16; ++np) {
      const uint32_t d = np * 16 + (lane >> 4) * 8;
      uint32_t r[4];
      ldmatrix_x4_t(r, base + (d / 64) * C::kBox + swz<C::kBoxBytes>(tok, (d % 64) * 2));
      add(2 * np, r[0], r[1]);
      add(2 * np + 1, r[2], r[3]);
    }
  } else {
    // Thread (g, q) holds the D / 8 elements from g D / 8 on of the tokens
    // 2q, 2q+1, 2q+8, 2q+9: column g of n-tile nt is element g D / 8 + nt.
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {     // eight elements at a time
      uint2 w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t tok = 2 * q + (t & 1) + (t >> 1) * 8;
        w[t] = *reinterpret_cast<const uint2*>(vs + swz<C::kBoxBytes>(tok, g * (D / 8) + c * 8));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t x = i == 0 ? w[t].x : w[t].y;
          lo[t] = e4m3x2_to_f16x2(x), hi[t] = e4m3x2_to_f16x2(x >> 16);
        }
        const int nt = 8 * c + 4 * i;
        add(nt + 0, __byte_perm(lo[0], lo[1], 0x5410), __byte_perm(lo[2], lo[3], 0x5410));
        add(nt + 1, __byte_perm(lo[0], lo[1], 0x7632), __byte_perm(lo[2], lo[3], 0x7632));
        add(nt + 2, __byte_perm(hi[0], hi[1], 0x5410), __byte_perm(hi[2], hi[3], 0x5410));
        add(nt + 3, __byte_perm(hi[0], hi[1], 0x7632), __byte_perm(hi[2], hi[3], 0x7632));
      }
    }
  }
}

// zero the value rows [from, kUnit) of a unit (whole warp)
template <int D, bool E4>
__device__ __forceinline__ void dec_zero_rows(uint8_t* vs, int from, int lane) {
  using C = DecCfg<D, E4>;
  constexpr int per_row = C::kRowBytes / 16;
  const int n = (C::kUnit - from) * per_row;
  for (int i = lane; i < n; i += 32) {
    const int row = from + i / per_row, c = i % per_row;
    const int box = c / (C::kBoxBytes / 16), cc = c % (C::kBoxBytes / 16);
    *reinterpret_cast<uint4*>(vs + box * C::kBox + row * C::kBoxBytes + cc * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();   // the slot's next TMA copy comes after these stores
  __syncwarp();
}

__device__ __forceinline__ bool word_nonfinite(uint32_t v, bool e4) {
  if (e4) return ((v & 0x7F) == 0x7F) | ((v & 0x7F00) == 0x7F00) | ((v & 0x7F0000) == 0x7F0000) |
                 ((v & 0x7F000000) == 0x7F000000);
  return ((v & 0x7F80) == 0x7F80) | ((v & 0x7F800000) == 0x7F800000);
}

// whether the value rows [from, to) of a unit hold a NaN or an infinity (whole warp)
template <int D, bool E4>
__device__ __forceinline__ bool dec_rows_nonfinite(const uint8_t* vs, int from, int to, int lane) {
  using C = DecCfg<D, E4>;
  constexpr int per_row = C::kRowBytes / 16;
  bool nf = false;
  for (int i = lane; i < (to - from) * per_row; i += 32) {
    const int row = from + i / per_row, c = i % per_row;
    const int box = c / (C::kBoxBytes / 16), cc = c % (C::kBoxBytes / 16);
    const uint4 v = *reinterpret_cast<const uint4*>(vs + box * C::kBox + row * C::kBoxBytes + cc * 16);
    nf |= word_nonfinite(v.x, E4) | word_nonfinite(v.y, E4) | word_nonfinite(v.z, E4) | word_nonfinite(v.w, E4);
  }
  return __any_sync(0xffffffffu, nf);
}

template <int D, bool E4>
__global__ void __launch_bounds__(kDecThreads, 2) attn_decode_kernel(const __grid_constant__ DecParams p) {
  using C = DecCfg<D, E4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* meet = reinterpret_cast<float*>(smem + C::kSlots * C::kSlotBytes);
  float* ml = meet + C::kMeet / 4;                 // [4][16][2] maximum and sum of each warp's rows
  float* fac = ml + kDecWarps * kDecRows * 2;      // [16][16] factors of the warps' outputs, of a join's first pieces
  float* row_m = fac + kDecJoin * kDecRows;        // [16] maximum and sum of the rows
  float* row_l = row_m + kDecRows;
  uint64_t* full = reinterpret_cast<uint64_t*>(row_l + kDecRows);
  uint64_t* empty = full + C::kSlots;
  uint64_t* meet_full = empty + C::kSlots;
  uint64_t* meet_free = meet_full + 1;
  uint64_t* piece_full = meet_free + 1;            // [pieces] told
  uint64_t* piece_empty = piece_full + kDecPieces; // [pieces] read by every other warp
  volatile int* told = reinterpret_cast<volatile int*>(piece_empty + kDecPieces);
  volatile int* abort_flag = told + kDecPieces * kDecPieceInts;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], C::kPerSlot);
    }
    mbar_init(meet_full, kDecWarps);
    mbar_init(meet_free, 1);
    for (int i = 0; i < kDecPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], kDecWarps + 1);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
  }
  __syncthreads();
  pdl_wait_primary();
  // (after the wait: whoever starts now finds the kernels before this one
  // complete. The tile kernel of the same call does not read what this one
  // writes; any other dependent waits for its completion.)
  pdl_allow_dependents();

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

  // the next piece, as the other warps get it; false: no more
  uint32_t told_n = 0;
  auto next_piece = [&](DecPiece& q) {
    const int e = told_n % kDecPieces;
    if (!wait(&piece_full[e], (told_n / kDecPieces) & 1u)) return false;
    int* to = reinterpret_cast<int*>(&q);
#pragma unroll
    for (int i = 0; i < kDecPieceInts; ++i) to[i] = told[e * kDecPieceInts + i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[e]);
    ++told_n;
    return q.t1 > q.t0;
  };

  if (warp == kDecWarps) {
    // ===== copying warp =====
    fence_proxy_async_global();
    DecWalk w;
    bool more = dec_begin<C::kTile>(p, w, lane);
    int slot = 0;
    uint32_t phase = 0;
    bool stop = false;
    while (!stop) {
      {
        const int e = told_n % kDecPieces;
        DecPiece q{};
        if (more) q = dec_piece_of(w);
        if (!wait(&piece_empty[e], ((told_n / kDecPieces) & 1u) ^ 1u)) break;
        if (lane == 0) {
          const int* from = reinterpret_cast<const int*>(&q);
#pragma unroll
          for (int i = 0; i < kDecPieceInts; ++i) told[e * kDecPieceInts + i] = from[i];
          mbar_arrive(&piece_full[e]);
        }
        __syncwarp();
        ++told_n;
        if (!more) break;
      }
      const int per = kDecGroup / p.box_rows;                       // boxes per slot
      const int boxes = (w.s.len + p.box_rows - 1) / p.box_rows;    // boxes that hold a token
      const int u0 = w.t0 * (C::kTile / kDecGroup) * per, u1 = w.t1 * (C::kTile / kDecGroup) * per;
      const int32_t* table = p.b.page_table + w.b * p.b.table_stride;
      auto page_of = [&](int u) {
        return u < min(boxes, u1) ? table[(u * p.box_rows) >> p.page_shift] : 0;
      };
      int pages = page_of(u0 + lane);
      for (int c = u0; c < u1 && !stop; c += 32) {
        const int now = pages;
        pages = page_of(c + 32 + lane);
        if (now < 0 || now >= p.num_pages) record_status(p.status, EPILORA_ERR_INVALID_ARG);
        const int n = min(32, u1 - c);
        for (int i = 0; i < n; i += per) {
          const int pg0 = __shfl_sync(0xffffffffu, now, i), pg1 = __shfl_sync(0xffffffffu, now, i + per - 1);
          if (!wait(&empty[slot], phase ^ 1u)) {
            stop = true;
            break;
          }
          if (elect_one()) {
            const int held = min(max(boxes - (c + i), 0), per);
            uint8_t* dst = smem + slot * C::kSlotBytes;
            if (held > 0)
              mbar_arrive_expect_tx(&full[slot], 2 * C::kRowBytes * held * p.box_rows);
            else
              mbar_arrive(&full[slot]);
            for (int k = 0; k < held; ++k) {
              const int row = ((c + i + k) * p.box_rows) & (p.page_size - 1);
              uint8_t* at = dst + k * p.box_rows * C::kBoxBytes;
#pragma unroll
              for (int x = 0; x < C::kBoxes; ++x) {
                // a page index out of range reads as zeros
                tma_load_4d(at + x * C::kBox, &p.tk, &full[slot], x * C::kBoxBytes, row, w.h, k ? pg1 : pg0);
                tma_load_4d(at + C::kHalf + x * C::kBox, &p.tv, &full[slot], x * C::kBoxBytes, row, w.h, k ? pg1 : pg0);
              }
            }
          }
          __syncwarp();
          if (++slot == C::kSlots) slot = 0, phase ^= 1u;
        }
      }
      more = dec_next<C::kTile>(p, w);
    }
    if (lane == 0) {
      // no copy in flight at exit (only after a wait that ran out is there
      // one that no computing warp has waited for): wait for the slots'
      // latest phases
      if (*abort_flag) {
        for (int i = 0; i < C::kSlots; ++i) {
          const uint32_t ph = i < slot ? phase : phase ^ 1u;
          (void)mbar_wait_bounded(&full[i], ph, 1000000ull);
        }
      }
    }
    return;
  }

  if (warp == kDecWarps + 1) {
    // ===== joining warp =====
    // packed rows of no sequence are zero
    {
      const int used = p.b.n_seqs > 0 ? min(max(p.b.q_start[p.b.n_seqs], 0), p.b.n_tokens) : 0;
      const int64_t rows = static_cast<int64_t>(p.b.n_tokens - used) * p.heads;
      constexpr int V = D / 8;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane; i < rows * V;
           i += static_cast<int64_t>(gridDim.x) * 32) {
        const int64_t r = i / V;
        const int64_t t = used + r / p.heads;
        const int h = static_cast<int>(r % p.heads);
        *reinterpret_cast<uint4*>(p.o.p + t * p.o.ts + h * p.o.hs + (i % V) * 8) = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr && i % V == 0) p.lse[t * p.heads + h] = -INFINITY;
      }
    }
    uint32_t piece = 0;
    DecPiece w;
    while (next_piece(w)) {
      if (!wait(meet_full, piece & 1u)) break;
      ++piece;
      const int rows = w.n * p.group;
      // lane 2 row + i: the warps' factors of a row, its maximum and sum
      float top = -INFINITY, sum = 0.0f;
      {
        const int row = lane >> 1;
#pragma unroll
        for (int k = 0; k < kDecWarps; ++k) top = fmaxf(top, ml[(k * kDecRows + row) * 2]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int k = 0; k < kDecWarps; ++k) {
          const float f = exp2_approx(ml[(k * kDecRows + row) * 2] - base);
          sum += ml[(k * kDecRows + row) * 2 + 1] * f;
          if ((k & 1) == (lane & 1)) fac[k * kDecRows + row] = f;
        }
        if (lane & 1) row_m[row] = top, row_l[row] = sum;
      }
      __syncwarp();
      const float vscale = E4 ? p.v_scale[w.h] : 1.0f;
      // four outputs of a row from element d on; m, l: the row's maximum and sum
      auto put = [&](int row, int d, float4 o, float m, float l) {
        const int i = row / p.group, h = w.h * p.group + row % p.group;
        const int64_t tok = w.first + i;
        const float inv = vscale / l;
        uint2 v = make_uint2(0, 0);   // (l == 0: the row sees nothing)
        if (l != 0.0f) v = make_uint2(pack16<false>(o.x * inv, o.y * inv), pack16<false>(o.z * inv, o.w * inv));
        *reinterpret_cast<uint2*>(p.o.p + tok * p.o.ts + h * p.o.hs + d) = v;
        if (p.lse != nullptr && d == 0)
          p.lse[tok * p.heads + h] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
      };
      const bool whole = w.whole != 0;
      constexpr int kPart = 2 * kDecRows + kDecRows * D;   // floats of a partial result: m, l, O
      constexpr int kMany = 4;
      float* part = p.partials + static_cast<int64_t>(w.slot) * kPart;
      // kMany elements a lane at a time: their loads run side by side
      for (int e0 = lane; e0 < rows * (D / 4); e0 += 32 * kMany) {
        float4 o[kMany];
#pragma unroll
        for (int y = 0; y < kMany; ++y) {
          const int row = (e0 + 32 * y) / (D / 4) & (kDecRows - 1), d = 4 * ((e0 + 32 * y) % (D / 4));
          o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < kDecWarps; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(meet + (k * kDecRows + row) * C::kOld + d);
            const float f = fac[k * kDecRows + row];
            o[y].x += v.x * f, o[y].y += v.y * f, o[y].z += v.z * f, o[y].w += v.w * f;
          }
        }
#pragma unroll
        for (int y = 0; y < kMany; ++y) {
          const int e = e0 + 32 * y, row = e / (D / 4) & (kDecRows - 1), d = 4 * (e % (D / 4));
          if (e >= rows * (D / 4)) continue;
          if (whole)
            put(row, d, o[y], row_m[row], row_l[row]);
          else
            *reinterpret_cast<float4*>(part + 2 * kDecRows + row * D + d) = o[y];
        }
      }
      if (!whole && (lane & 1) == 0) part[lane >> 1] = top, part[kDecRows + (lane >> 1)] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(meet_free);
      if (whole) continue;
      const int first = w.first_cta, pieces = w.pieces;
      uint32_t is_last = 0;
      if (lane == 0) {
        // (the warp's stores are before it: the barrier above)
        is_last = atom_inc_acq_rel_gpu(p.counters + first) == static_cast<uint32_t>(pieces - 1);
        if (is_last) p.counters[first] = 0;
      }
      if (!__shfl_sync(0xffffffffu, is_last, 0)) continue;
      auto piece_at = [&](int k) {
        return p.partials + static_cast<int64_t>(k == 0 ? w.slot0 : 2 * (first + k)) * kPart;
      };
      // Maximum and sum of row lane / 2 over the pieces, of which this lane
      // takes every other one; the first 16 pieces' loads are under way at once.
      const int my_row = lane >> 1, odd = lane & 1;
      float pm[kDecJoin / 2], pl[kDecJoin / 2];
#pragma unroll
      for (int i = 0; i < kDecJoin / 2; ++i) {
        const int k = 2 * i + odd;
        pm[i] = k < pieces ? __ldcg(piece_at(k) + my_row) : -INFINITY;
        pl[i] = k < pieces ? __ldcg(piece_at(k) + kDecRows + my_row) : 0.0f;
      }
      top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kDecJoin / 2; ++i) top = fmaxf(top, pm[i]);
      for (int k = kDecJoin + odd; k < pieces; k += 2) top = fmaxf(top, __ldcg(piece_at(k) + my_row));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int i = 0; i < kDecJoin / 2; ++i) {
        pm[i] = exp2_approx(pm[i] - base);
        sum += pl[i] * pm[i];
        fac[(2 * i + odd) * kDecRows + my_row] = pm[i];
      }
      for (int k = kDecJoin + odd; k < pieces; k += 2)
        sum += __ldcg(piece_at(k) + kDecRows + my_row) * exp2_approx(__ldcg(piece_at(k) + my_row) - base);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      if (odd) row_m[my_row] = top, row_l[my_row] = sum;
      __syncwarp();
      for (int e0 = lane; e0 < rows * (D / 4); e0 += 32 * kMany) {
        float4 o[kMany];
#pragma unroll
        for (int y = 0; y < kMany; ++y) o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = 0; k0 < min(pieces, kDecJoin); k0 += 4) {
          float4 v[4][kMany];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < kMany; ++y) {
              const int e = e0 + 32 * y;     // (element e of the rows is float4 e of the piece's outputs)
              v[i][y] = k0 + i < pieces && e < rows * (D / 4)
                            ? __ldcg(reinterpret_cast<const float4*>(piece_at(k0 + i) + 2 * kDecRows) + e)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < kMany; ++y) {
              const float f = fac[(k0 + i) * kDecRows + ((e0 + 32 * y) / (D / 4) & (kDecRows - 1))];
              o[y].x += v[i][y].x * f, o[y].y += v[i][y].y * f, o[y].z += v[i][y].z * f, o[y].w += v[i][y].w * f;
            }
        }
#pragma unroll
        for (int y = 0; y < kMany; ++y) {
          const int e = e0 + 32 * y, row = e / (D / 4), d = 4 * (e % (D / 4));
          if (e >= rows * (D / 4)) continue;
          const float m = row_m[row], row_base = m == -INFINITY ? 0.0f : m;
          for (int k = kDecJoin; k < pieces; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(piece_at(k) + 2 * kDecRows) + e);
            const float f = exp2_approx(__ldcg(piece_at(k) + row) - row_base);
            o[y].x += v.x * f, o[y].y += v.y * f, o[y].z += v.z * f, o[y].w += v.w * f;
          }
          put(row, d, o[y], m, row_l[row]);
        }
      }
      __syncwarp();     // the factors are free again
    }
    return;
  }

  // ===== computing warps =====
  const int g = lane >> 2, q = lane & 3;
  int slot = warp / C::kPerSlot;
  uint32_t piece = 0;
  uint32_t phase = 0;
  bool dead = false;
  DecPiece w;
  while (!dead && next_piece(w)) {
    const int n = w.n, rows = n * p.group;
    // the thread's two rows: token i, head, positions it sees
    const int r0 = g, r1 = g + 8;
    const int i0 = r0 / p.group, i1 = r1 / p.group;
    const bool ok0 = r0 < rows, ok1 = r1 < rows;
    const int see0 = ok0 ? max(min(w.base + i0 + 1, w.len), 0) : 0;
    const int see1 = ok1 ? max(min(w.base + i1 + 1, w.len), 0) : 0;
    const int see_all = max(min(w.base + 1, w.len), 0);    // positions every row sees
    float s_eff = p.scale;
    if (E4) s_eff *= p.k_scale[w.h];
    const uint32_t flip = s_eff < 0.0f ? 0x80008000u : 0u;
    float c0 = s_eff == 0.0f ? 1.0f : fabsf(s_eff) * kLog2e, c1 = c0;

    // Q fragments
    uint32_t qa[D / 16][4];
    {
      const __nv_bfloat16* q0 = p.q.p + (w.first + i0) * p.q.ts + (w.h * p.group + r0 % p.group) * p.q.hs;
      const __nv_bfloat16* q1 = p.q.p + (w.first + i1) * p.q.ts + (w.h * p.group + r1 % p.group) * p.q.hs;
      const bool zero = s_eff == 0.0f;
      if (!E4) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int d = ks * 16 + 2 * q;
          qa[ks][0] = ok0 && !zero ? *reinterpret_cast<const uint32_t*>(q0 + d) ^ flip : 0u;
          qa[ks][1] = ok1 && !zero ? *reinterpret_cast<const uint32_t*>(q1 + d) ^ flip : 0u;
          qa[ks][2] = ok0 && !zero ? *reinterpret_cast<const uint32_t*>(q0 + d + 8) ^ flip : 0u;
          qa[ks][3] = ok1 && !zero ? *reinterpret_cast<const uint32_t*>(q1 + d + 8) ^ flip : 0u;
        }
      } else {
        // fp16 queries: bf16's 8 significant bits fit; each row is scaled by
        // the power of two that puts its largest element near 2^13 (elements
        // 2^27 below that are still exact, the rest is off by 2^-38 of the
        // largest), the scores' factor takes it back
        uint4 raw[2][D / 64][2];
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = 64 * c + 16 * q + 8 * e;
            raw[0][c][e] = ok0 && !zero ? *reinterpret_cast<const uint4*>(q0 + d) : make_uint4(0, 0, 0, 0);
            raw[1][c][e] = ok1 && !zero ? *reinterpret_cast<const uint4*>(q1 + d) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float big = 0.0f;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 v = raw[r][c][e];
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k]))));
            }
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // 2^(13 - exponent), within the normal range; 1 for rows of zeros
          // or with an infinity
          const int ex = static_cast<int>((__float_as_uint(big) >> 23) & 0xFF);
          const int up = big == 0.0f || ex == 0xFF ? 0 : min(13 - (ex - 127), 126);
          const float f = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
          (r == 0 ? c0 : c1) *= up == 0 ? 1.0f : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 v = raw[r][c][j >> 1];
              const uint32_t a = (j & 1) ? v.z : v.x, b = (j & 1) ? v.w : v.y;
              qa[4 * c + j][r] = pack16<true>(bf16_lo(a) * f, bf16_hi(a) * f) ^ flip;
              qa[4 * c + j][2 + r] = pack16<true>(bf16_lo(b) * f, bf16_hi(b) * f) ^ flip;
            }
        }
      }
    }

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;

    for (int t = w.t0; t < w.t1; ++t) {
      const int at = t * C::kTile + warp * C::kUnit;
      if (!dead) dead = !wait(&full[slot], phase);
      if (!dead && at < w.len) {
        uint8_t* ks = smem + slot * C::kSlotBytes + (warp % C::kPerSlot) * C::kUnitBytes;
        uint8_t* vs = ks + C::kHalf;
        // rows of the page that hold no token of this sequence
        if (at + C::kUnit > w.len) dec_zero_rows<D, E4>(vs, w.len - at, lane);
        constexpr int NT = C::kUnit / 8;      // columns of scores, eight positions each
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
        if (!E4) {
          const uint32_t base = smem_u32(ks);
          const uint32_t tok = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t d = k * 16 + ((lane >> 3) & 1) * 8;
            uint32_t r[4];
            ldmatrix_x4(r, base + (d / 64) * C::kBox + swz<C::kBoxBytes>(tok, (d % 64) * 2));
            mma16<E4>(s[0], qa[k], r[0], r[1]);
            mma16<E4>(s[1], qa[k], r[2], r[3]);
          }
        } else {
          // thread (g, q): elements 64 c + 16 q .. + 15 of the tokens 8 nt + g;
          // step j of a c contracts elements 4 j .. 4 j + 3 of each thread
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 v = *reinterpret_cast<const uint4*>(ks + swz<C::kBoxBytes>(nt * 8 + g, 64 * c + 16 * q));
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma16<E4>(s[nt], qa[4 * c + j], e4m3x2_to_f16x2(x[j]), e4m3x2_to_f16x2(x[j] >> 16));
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] *= c0, s[nt][1] *= c0;
          s[nt][2] *= c1, s[nt][3] *= c1;
        }
        const bool edge = at + C::kUnit > see_all;
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = at + nt * 8 + 2 * q + e;
              if (pos >= see0) s[nt][e] = -INFINITY;
              if (pos >= see1) s[nt][2 + e] = -INFINITY;
            }
        }
        float x0 = fmaxf(s[0][0], s[0][1]), x1 = fmaxf(s[0][2], s[0][3]);
#pragma unroll
        for (int nt = 1; nt < NT; ++nt) x0 = max3(x0, s[nt][0], s[nt][1]), x1 = max3(x1, s[nt][2], s[nt][3]);
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        // m: the running maximum less the lift
        constexpr float kLift = kWeightLift<E4>;
        const bool up0 = x0 > m0 + (kRaise + kLift), up1 = x1 > m1 + (kRaise + kLift);
        if (__any_sync(0xffffffffu, up0 || up1)) {
          x0 -= kLift, x1 -= kLift;
          const float f0 = up0 ? exp2_approx(m0 - x0) : 1.0f, f1 = up1 ? exp2_approx(m1 - x1) : 1.0f;
          if (up0) m0 = x0;
          if (up1) m1 = x1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) acc[i][0] *= f0, acc[i][1] *= f0, acc[i][2] *= f1, acc[i][3] *= f1;
        }
        const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
        uint32_t pa[NT / 2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] = exp2_approx(s[nt][0] - b0), s[nt][1] = exp2_approx(s[nt][1] - b0);
          s[nt][2] = exp2_approx(s[nt][2] - b1), s[nt][3] = exp2_approx(s[nt][3] - b1);
          l0 += s[nt][0] + s[nt][1];
          l1 += s[nt][2] + s[nt][3];
          // the weights as 16-bit operands (each within 2^-8 of itself in bf16; fp16: see kWeightLift)
          pa[nt / 2][2 * (nt & 1)] = pack16<E4>(s[nt][0], s[nt][1]);
          pa[nt / 2][2 * (nt & 1) + 1] = pack16<E4>(s[nt][2], s[nt][3]);
        }
        // A zero weight times a NaN or an infinity is NaN: where a position
        // is hidden from some rows and holds one, each token's rows take
        // their own product, the later positions zeroed from the last token
        // to the first.
        if (edge && n > 1 && dec_rows_nonfinite<D, E4>(vs, max(see_all - at, 0), min(C::kUnit, w.len - at), lane)) {
#pragma unroll 1
          for (int i = n - 1; i >= 0; --i) {
            const int see = max(min(w.base + i + 1, w.len), 0) - at;
            if (see < C::kUnit) dec_zero_rows<D, E4>(vs, max(see, 0), lane);
#pragma unroll
            for (int u = 0; u < NT / 2; ++u)
              dec_pv<D, E4, true>(acc, pa[u], vs + u * 16 * C::kBoxBytes, lane, ok0 && i0 == i, ok1 && i1 == i);
          }
        } else {
#pragma unroll
          for (int u = 0; u < NT / 2; ++u)
            dec_pv<D, E4, false>(acc, pa[u], vs + u * 16 * C::kBoxBytes, lane, true, true);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      slot += C::kSlotStep;
      if (slot >= C::kSlots) slot -= C::kSlots, phase ^= 1u;
    }

    // ===== handed to the joining warp =====
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // (after a wait that ran out nothing is waited for any more)
    if (!dead) dead = !wait(meet_free, (piece & 1u) ^ 1u);
    ++piece;
    if (q == 0) {
      ml[(warp * kDecRows + r0) * 2] = m0, ml[(warp * kDecRows + r0) * 2 + 1] = l0;
      ml[(warp * kDecRows + r1) * 2] = m1, ml[(warp * kDecRows + r1) * 2 + 1] = l1;
    }
    float* mine = meet + warp * kDecRows * C::kOld;
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt) {
      // columns 2q and 2q + 1 of n-tile nt
      const int d0 = E4 ? 2 * q * (D / 8) + nt : nt * 8 + 2 * q;
      const int d1 = E4 ? d0 + D / 8 : d0 + 1;
      if (ok0) mine[r0 * C::kOld + d0] = acc[nt][0], mine[r0 * C::kOld + d1] = acc[nt][1];
      if (ok1) mine[r1 * C::kOld + d0] = acc[nt][2], mine[r1 * C::kOld + d1] = acc[nt][3];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(meet_full);
  }
}

template <int D, bool E4>
int launch(const AttnArgs& a, DecParams& p, int grid) {
  using C = DecCfg<D, E4>;
  const epilora_kv_cache& c = a.cache;
  const uint64_t es = E4 ? 1 : 2;
  const uint64_t dims[4] = {static_cast<uint64_t>(C::kRowBytes), static_cast<uint64_t>(c.page_size),
                            static_cast<uint64_t>(c.kv_heads), static_cast<uint64_t>(c.num_pages)};
  const uint32_t box[4] = {static_cast<uint32_t>(C::kBoxBytes), static_cast<uint32_t>(p.box_rows), 1, 1};
  const uint64_t ks[3] = {c.k_token_stride * es, c.k_head_stride * es, c.k_page_stride * es};
  const uint64_t vs[3] = {c.v_token_stride * es, c.v_head_stride * es, c.v_page_stride * es};
  int rc = make_tma_4d_u8(&p.tk, c.k, dims, ks, box, C::kBoxBytes);
  if (rc == EPILORA_OK) rc = make_tma_4d_u8(&p.tv, c.v, dims, vs, box, C::kBoxBytes);
  if (rc != EPILORA_OK) return rc;
  auto kern = attn_decode_kernel<D, E4>;
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EPILORA_ERR_CUDA;
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return EPILORA_ERR_CUDA;
    attr_done[dev] = 1;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kDecThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? EPILORA_OK : EPILORA_ERR_CUDA;
}

int dec_ctas() {
  const int n = 2 * num_sms();
  return n < kDecMaxCtas ? n : kDecMaxCtas;
}

}  // namespace

size_t attn_decode_counter_bytes() { return kDecMaxCtas * sizeof(uint32_t); }
size_t attn_decode_partial_bytes(int head_dim) {
  return static_cast<size_t>(2 * dec_ctas()) * (2 * kDecRows + kDecRows * head_dim) * sizeof(float);
}

int launch_attn_decode(const AttnArgs& a, uint32_t* counters, float* partials) {
  DecParams p{};
  p.b = a.batch;
  p.q = a.q;
  p.o = a.o;
  p.lse = a.lse;
  p.heads = a.heads;
  p.kv_heads = a.cache.kv_heads;
  p.group = a.heads / a.cache.kv_heads;
  p.page_shift = __builtin_ctz(a.cache.page_size);
  p.page_size = a.cache.page_size;
  p.num_pages = a.cache.num_pages;
  p.box_rows = a.cache.page_size < kDecGroup ? a.cache.page_size : kDecGroup;
  p.scale = a.scale;
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.counters = counters;
  p.partials = partials;
  p.status = a.status;
  // no more blocks than tiles there can be
  const bool e4 = a.cache.kv_fmt == EPILORA_KV_E4M3;
  const int tile = e4 ? DecCfg<128, true>::kTile : DecCfg<128, false>::kTile;
  const int64_t cap = static_cast<int64_t>(a.batch.table_pages) * a.cache.page_size;
  const int64_t most = a.batch.n_seqs * (a.cache.kv_heads * ((cap + tile - 1) / tile + 1));
  if (most >= (int64_t{1} << 32)) return EPILORA_ERR_UNSUPPORTED;    // the line's tiles are counted in 32 bits
  const int grid = static_cast<int>(most < 1 ? 1 : (most < dec_ctas() ? most : dec_ctas()));
  if (a.cache.head_dim == 64) return e4 ? launch<64, true>(a, p, grid) : launch<64, false>(a, p, grid);
  return e4 ? launch<128, true>(a, p, grid) : launch<128, false>(a, p, grid);
}

}  // namespace epi
