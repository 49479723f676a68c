// The block-scaled products of few rows (decoding): the product turned round,
// so that the weights are the rows of the MMA.
//
// What such a call has to do is to read the weights once. With rows of A as
// rows of the MMA (block_gemm.cu) a tile of few rows keeps 32 of 128 TMEM lanes
// busy, so one warp in four, with 128 columns each per block; here 128 rows of
// W fill the lanes, up to 32 rows of A are the columns, and all summing warps
// share the work: 16 products a thread and block. A half of TMEM then holds
// eight blocks, loaded together, so that a load's latency and the barriers are
// paid once for 128 KB of weights.
//
// Roles (384 threads, one CTA per SM):
//   warp 0       TMA copies through a ring of stages
//   warp 1       MMA issue (M = 128, N = 32)
//   warp 2       the scales of the groups to come
//   warps 4..11  sums: each warp 32 rows of W by half of the rows of A
// A plain product is split along K over the CTAs of a cluster (up to 8): each
// sends its sums to the CTA that finishes the row of A, which adds them in the
// order of the CTAs. Gated: a tile is 128 rows of gate and the same of up.
// In both the sums leave the registers for shared memory, and what follows is
// a loop over it: a tile is finished once or a few times per launch, when code
// that is unrolled over the registers comes from memory at some 500 cycles a
// line (the joined sums of 32 x 14336 -> 4096 took 7000 cycles to store).
//
// Bound: the copies of the weights, and start and end. Up projections of 64 tokens over 64 experts of 4096 x 1792 take
// 132 us with plan and scatter (7.1 TB/s of the experts' 940 MB: some of them stay in L2), of one token 29.5 us (117 MB);
// 32 x 14336 -> 4096 18.5 us with the quantizer (59 MB). Every wait is bounded, as in block_gemm.cu.
#include "block_gemm.cuh"

namespace epi {

namespace {

constexpr int kThreads = 384;
constexpr int kTileN = 128;                    // rows of W per tile
constexpr int kCols = 32;                      // rows of A per tile: columns of the MMA
constexpr int kHalf = 256;
constexpr int kWBytes = kTileN * kBlock, kABytes = kCols * kBlock;     // of a block
constexpr int kStagesMax = 12;
// registers: 168 a thread at launch (64,512); the sums' warps take what the others give back
constexpr int kRegsOther = 48, kRegsSum = 224;
constexpr int kScaleRow = kCols + 4;           // a block's scales: of the rows, then of the weights (gate, up)
constexpr int kScaleBlocks = 32;
constexpr int kMine = kCols / 2;               // rows of A of a summing thread
constexpr int kMisc = 1024 + kScaleBlocks * kScaleRow * 4;             // barriers, scales
// sums on their way: of the rows that this CTA finishes [CTA][row][kTileN] (as many rows times CTAs as there are columns);
// gated, [gate, up][kCols][kTileN]
template <bool kGated>
constexpr int kSumBytes = (kGated ? 2 : 1) * kCols * kTileN * 4;

struct Params {
  CUtensorMap tmA, tmB;
  const float* a_scale;
  const float* w_scale;
  int64_t a_scale_ld, ldy;
  void* Y;
  uint8_t* inner;
  float* inner_scale;
  const int32_t* offsets;
  const int32_t* out_rows;
  int* status;
  int M, N, kb, n_tiles, experts, stages, copy, whole, splits, early_weights;
  int late;                // the test hook: the copies of a tile's last stage never seem complete
};

// Gated products are of the rows by expert, others of plain matrices.
template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1) block_few_kernel(const __grid_constant__ Params p) {
  constexpr bool kGrouped = kGated;
  constexpr int kParts = kGated ? 2 : 1;       // gate, up
  constexpr int G = kHalf / (kCols * kParts);  // blocks of a group
  constexpr int kSlots = kScaleBlocks / G;     // groups in the scales' ring
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stages = p.stages, copy = kGated ? 1 : p.copy;
  const uint32_t stage = copy * (kParts * kWBytes + kABytes);      // the blocks' weights, then their rows of A
  uint8_t* misc = smem + static_cast<size_t>(stages) * stage;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + kStagesMax;
  uint64_t* filled = empty + kStagesMax;       // [2] a half holds a group's products, and the ring its scales
  uint64_t* drained = filled + 2;              // [2] they have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* scales = reinterpret_cast<float*>(misc + 1024);                   // [kScaleBlocks][kScaleRow]
  float* sums = reinterpret_cast<float*>(misc + kMisc);
  int* offsets = reinterpret_cast<int*>(misc + kMisc + kSumBytes<kGated>); // [experts + 1], grouped only
  int* starts = offsets + p.experts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kGrouped ? 0 : static_cast<int>(blockIdx.x) % p.splits;
  // this CTA's blocks of K
  const int k0 = kGrouped ? 0 : p.kb * rank / p.splits;
  const int kb = kGrouped ? p.kb : p.kb * (rank + 1) / p.splits - k0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&filled[b], 2);                // the products, and the scales
      mbar_init(&drained[b], 8);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kHalf);
    tmem_relinquish();
  }
  if (kGrouped) {
    pdl_wait_primary();
    if (warp == 2) fill_walk<kCols>(p.offsets, p.experts, offsets, starts, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!kGated) cluster_arrive();       // (waited for where sums are sent: every CTA has started by then)
  pdl_allow_dependents();
  const uint32_t tmem_base = *tmem_slot;
  Walk<kGrouped, kCols> walk(p.M, p.n_tiles, p.experts, offsets, starts);
  const int first_tile = static_cast<int>(blockIdx.x) / p.splits, step = static_cast<int>(gridDim.x) / p.splits;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag, p.status); };

  if (warp < 4) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == 0) {
      // ===== copies =====
      if (elect_one()) {
        int s = 0;
        uint32_t ph = 0, issued = 0, phases = 0;
        bool go = true, waited = kGrouped;
        if (kGrouped) fence_proxy_async_global();
        for (int t = first_tile; t < walk.total && go; t += step) {
          const Tile tile = walk.at(t);
          const int wrow = tile.expert * kParts * p.N + tile.n * kTileN;
          const auto load = [&](uint8_t* dst, const CUtensorMap* map, int st, int row, int b) {
            tma_load_4d(dst, map, &full[st], p.whole ? 0 : (k0 + b) * kBlock, row, p.whole ? k0 + b : 0, 0);
          };
          // (a stage that reaches past this CTA's blocks copies some that nobody uses)
          const auto copy_w = [&](int st, int b) {
            uint8_t* dst = smem + static_cast<size_t>(st) * stage;
            mbar_arrive_expect_tx(&full[st], stage + (p.late && b + copy >= kb ? 16 : 0));
            load(dst, &p.tmB, st, wrow, b);
            if (kGated) load(dst + kWBytes, &p.tmB, st, wrow + p.N, b);
          };
          int early = 0;
          if (!waited) {
            // weights of the first stages before the rows are there
            early = p.early_weights ? min(stages, (kb + copy - 1) / copy) : 0;
            for (int i = 0; i < early; ++i) copy_w(i, i * copy);
            issued |= (1u << early) - 1u;
            pdl_wait_primary();
            fence_proxy_async_global();
            waited = true;
          }
          for (int b = 0; b < kb; b += copy) {
            if (!wait(&empty[s], ph ^ 1u)) {
              go = false;
              break;
            }
            if (b >= early * copy) copy_w(s, b);
            load(smem + static_cast<size_t>(s) * stage + copy * kParts * kWBytes, &p.tmA, s, tile.first, b);
            issued |= 1u << s;
            phases = (phases & ~(1u << s)) | (ph << s);
            if (++s == stages) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        if (*abort_flag) {
          // no copy in flight at exit
          for (int i = 0; i < stages; ++i)
            if (issued & (1u << i)) (void)mbar_wait_bounded(&full[i], (phases >> i) & 1u, kWaitLimitNs);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ===== MMA issue =====
      pdl_wait_primary();      // (its first wait is for rows that the preceding kernels write, however long those take)
      if (elect_one()) {
        constexpr uint32_t kIdesc = idesc_f8f6f4_e4m3(kTileN, kCols);
        const uint64_t desc0 = make_smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        int s = 0, half = 0;
        uint32_t ph = 0, hph = 0;
        bool go = true, any = false;
        for (int t = first_tile; t < walk.total && go; t += step) {
          for (int b0 = 0; b0 < kb; b0 += G) {
            if (!wait(&drained[half], hph ^ 1u)) {
              go = false;
              break;
            }
            const int n = min(G, kb - b0);
            for (int u = 0; u < n; ++u) {
              const int i = (b0 + u) & (copy - 1);      // of the stage's blocks
              if (i == 0 && !wait(&full[s], ph)) {
                go = false;
                break;
              }
              tc_fence_after();
              // (descriptors count 16 bytes: 2 more for each 32 bytes of K)
              const uint64_t wd = desc0 + ((s * stage + i * kParts * kWBytes) >> 4);
              const uint64_t ad = desc0 + ((s * stage + copy * kParts * kWBytes + i * kABytes) >> 4);
              const uint32_t d = tmem_base + half * kHalf + u * kCols * kParts;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int part = 0; part < kParts; ++part)
                  mma_f8f6f4(d + part * kCols, wd + part * (kWBytes >> 4) + 2 * kk, ad + 2 * kk, kIdesc, kk > 0);
              if (i == copy - 1 || b0 + u == kb - 1) {
                tc_commit(&empty[s]);
                any = true;
                if (++s == stages) {
                  s = 0;
                  ph ^= 1u;
                }
              }
            }
            if (!go) break;        // (a group that is not whole is handed to nobody)
            tc_commit(&filled[half]);
            half ^= 1;
            if (half == 0) hph ^= 1u;
          }
        }
        // nothing of this thread in flight at exit: the last stage's commit covers every MMA before it
        if (any) (void)mbar_wait_bounded(&empty[s > 0 ? s - 1 : stages - 1], s > 0 ? ph : ph ^ 1u, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ===== scales =====
      constexpr int kAhead = kSlots - 2;         // groups under way (the slot before the last one may be read still)
      const int nb = n_blocks(p.N);
      pdl_wait_primary();
      Walk<kGrouped, kCols> ahead = walk;
      int c_t = first_tile, c_b = 0, put = 0;
      Tile tile{};
      const float *c_a = nullptr, *c_w = nullptr;
      const auto enter = [&] {
        tile = ahead.at(c_t);
        c_a = p.a_scale + tile.first + lane + k0 * p.a_scale_ld;
        c_w = p.w_scale + static_cast<int64_t>((tile.expert * kParts + (lane & (kParts - 1))) * nb + tile.n) * p.kb + k0;
      };
      const auto fetch = [&] {
        if (c_t < ahead.total) {
          float* slot = scales + put * (G * kScaleRow);
          const int n = min(G, kb - c_b);
          for (int u = 0; u < n; ++u) {
            if (lane < tile.rows) copy4(slot + u * kScaleRow + lane, c_a + (c_b + u) * p.a_scale_ld);
            if (lane < kParts) copy4(slot + u * kScaleRow + kCols + lane, c_w + c_b + u);
          }
          put = (put + 1) & (kSlots - 1);
          c_b += G;
          if (c_b >= kb) {
            c_b = 0;
            c_t += step;
            if (c_t < ahead.total) enter();
          }
        }
        copies_commit();
      };
      if (c_t < ahead.total) enter();
  #pragma unroll 1
      for (int g = 0; g < kAhead; ++g) fetch();
      int half = 0;
      uint32_t hph = 0;
      bool go = true;
      for (int t = first_tile; t < walk.total && go; t += step)
        for (int b0 = 0; b0 < kb; b0 += G) {
          go = __all_sync(0xffffffffu, wait(&drained[half], hph ^ 1u));
          if (!go) break;
          fetch();
          copies_wait<kAhead>();
          __syncwarp();
          if (lane == 0) mbar_arrive(&filled[half]);
          half ^= 1;
          if (half == 0) hph ^= 1u;
        }
      copies_wait<0>();
    }
    if (!kGated) {
      // the cluster's barriers (see the sums) count every thread
      __syncwarp();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
  } else {
    // ===== sums =====
    setmaxnreg_inc<kRegsSum>();
    pdl_wait_primary();
    const int side = (warp - 4) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;            // of the tile's rows of W
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + side * kMine;
    int half = 0, take = 0;
    uint32_t hph = 0;
    bool dead = false;
    for (int t = first_tile; t < walk.total; t += step) {
      const Tile tile = walk.at(t);
      const int mine = min(tile.rows - side * kMine, kMine);       // rows of A of this side
      const float start = dead ? __int_as_float(0x7fffffff) : 0.0f;
      float acc[kParts][kMine];
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int c = 0; c < kMine; ++c) acc[part][c] = start;
#pragma unroll 1
      for (int b0 = 0; b0 < kb; b0 += G) {
        if (!dead && !__all_sync(0xffffffffu, wait(&filled[half], hph))) dead = true;
        if (!dead) {
          tc_fence_after();
          const int blocks = min(G, kb - b0);
          const float* sc = scales + take * (G * kScaleRow) + side * kMine;
          uint32_t v[G * kParts][kMine];
          if (mine > 0) {
#pragma unroll
            for (int i = 0; i < G * kParts; ++i)
              if (i < kParts * blocks) tmem_ld_32x32b_x16(lanes + half * kHalf + i * kCols, v[i]);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < G; ++u)
              if (u < blocks) {
                const float* row = sc + u * kScaleRow;
                float as[kMine];
#pragma unroll
                for (int c = 0; c < kMine; c += 4) {
                  const float4 q = *reinterpret_cast<const float4*>(row + c);
                  as[c] = q.x, as[c + 1] = q.y, as[c + 2] = q.z, as[c + 3] = q.w;
                }
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                  const float ws = row[kCols - side * kMine + part];
#pragma unroll
                  for (int c = 0; c < kMine; ++c)
                    asm volatile("fma.rn.f32 %0, %1, %2, %0;"      // (volatile: behind the wait for the loads)
                                 : "+f"(acc[part][c])
                                 : "f"(__uint_as_float(v[u * kParts + part][c])), "f"(as[c] * ws));
                }
              }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&drained[half]);
        }
        take = (take + 1) & (kSlots - 1);
        half ^= 1;
        if (half == 0) hph ^= 1u;
      }
      if (dead && start == 0.0f) {     // sums that are not whole: the tile once more, as NaN (others finish them too)
        t -= step;
        continue;
      }
      const int me = static_cast<int>(threadIdx.x) - 128;
      if constexpr (kGated) {
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int c = 0; c < kMine; ++c) sums[(part * kCols + side * kMine + c) * kTileN + r] = acc[part][c];
        asm volatile("bar.sync 1, 256;" ::: "memory");
        // a warp a row of A, a lane four elements of its block
        const int n = tile.n * kTileN + lane * 4;
#pragma unroll 1
        for (int c = warp - 4; c < tile.rows; c += 8) {
          const float4 g = *reinterpret_cast<const float4*>(sums + c * kTileN + lane * 4);
          const float4 u = *reinterpret_cast<const float4*>(sums + (kCols + c) * kTileN + lane * 4);
          // (a width that is a multiple of 16 has all four or none)
          const bool there = n < p.N;
          const float h[4] = {there ? silu(g.x) * u.x : 0.0f, there ? silu(g.y) * u.y : 0.0f,
                              there ? silu(g.z) * u.z : 0.0f, there ? silu(g.w) * u.w : 0.0f};
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(h[i]));
          const float s = block_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
          const BlockDiv by = block_div(s);
          float d[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = div_rn_by_recip(h[i], by.s, by.rs);
          const int64_t to = p.out_rows != nullptr ? __ldcg(p.out_rows + tile.first + c) : tile.first + c;
          if (there)
            *reinterpret_cast<uint32_t*>(p.inner + to * p.N + n) = cvt_e4m3x2(d[0], d[1]) | (cvt_e4m3x2(d[2], d[3]) << 16);
          if (lane == 0) p.inner_scale[static_cast<int64_t>(tile.n) * p.M + to] = s;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");       // (the next tile's sums)
      } else {
        // row c of A is finished by CTA c / per of the cluster
        const int per = kCols / p.splits;
        cluster_wait();
#pragma unroll
        for (int c = 0; c < kMine; ++c) {
          const int row = side * kMine + c;
          st_dsmem_f32(map_to_cta(smem_u32(sums + (rank * per + row % per) * kTileN + r), row / per), acc[0][c]);
        }
        cluster_arrive();
        cluster_wait();
#pragma unroll 1
        for (int i = me; i < per * kTileN; i += 256) {
          const int row = rank * per + i / kTileN, n = tile.n * kTileN + i % kTileN;
          float y = sums[i];
          for (int q = 1; q < p.splits; ++q) y += sums[q * per * kTileN + i];
          if (row < tile.rows && n < p.N)
            static_cast<__nv_bfloat16*>(p.Y)[(tile.first + row) * p.ldy + n] = __float2bfloat16_rn(y);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kHalf);
  }
}

// A tensor map of a matrix [rows][K] of bytes whose copies take `copy` blocks of K of `box_rows` rows each: 128 bytes,
// rows, blocks. Where K ends inside a block there is no axis of blocks (the last one would run into the next row), and
// a copy takes one, at its place in the row.
int make_tma_blocks(CUtensorMap* map, const void* base, int64_t rows, int K, int box_rows, int copy) {
  const bool whole = K % kBlock == 0;
  const uint64_t row = static_cast<uint64_t>(K), n = static_cast<uint64_t>(rows);
  const uint64_t dims[4] = {whole ? kBlock : row, n, whole ? row / kBlock : 1, 1};
  const uint64_t strides[3] = {row, whole ? kBlock : row, row};
  const uint32_t box[4] = {kBlock, static_cast<uint32_t>(box_rows), static_cast<uint32_t>(copy), 1};
  return make_tma_4d_u8(map, base, dims, strides, box, 128);
}

// CTAs that share K: as many as still find an SM each (of clusters of 2, 4 and 8 this GPU runs 76, 36 and 15 at once),
// while each keeps a group of blocks.
int few_splits(int N, int K) {
  const int n_tiles = (N + kTileN - 1) / kTileN, most[3] = {76, 36, 15};
  int splits = 1;
  for (int i = 0; i < 3 && n_tiles <= most[i] && n_blocks(K) >= 8 * 2 * splits; ++i) splits *= 2;
  return splits;
}

template <bool kGated>
int launch(const BlockGemmArgs& a) {
  constexpr bool kGrouped = kGated;
  Params p{};
  p.a_scale = a.a_scale;
  p.w_scale = a.w_scale;
  p.a_scale_ld = a.a_scale_ld;
  p.Y = a.Y;
  p.ldy = a.ldy;
  p.inner = a.inner;
  p.inner_scale = a.inner_scale;
  p.offsets = a.offsets;
  p.out_rows = a.out_rows;
  p.status = a.status;
  p.M = a.M;
  p.N = a.N;
  p.kb = n_blocks(a.K);
  p.experts = kGrouped ? a.experts : 1;
  p.early_weights = a.early_weights;
  p.late = block_test_late_copies();
  p.n_tiles = (a.N + kTileN - 1) / kTileN;
  p.whole = a.K % kBlock == 0;
  p.copy = kGated || !p.whole ? 1 : 2;         // 40 KB a stage, five stages
  const int64_t w_rows = static_cast<int64_t>(p.experts) * a.N * (kGated ? 2 : 1);
  const int64_t tiles = (static_cast<int64_t>(a.M) / kCols + 1 + (kGrouped ? p.experts : 0)) * p.n_tiles;
  if (tiles > EPILORA_BLOCK_MAX_SIZE || w_rows > EPILORA_BLOCK_MAX_SIZE) return EPILORA_ERR_UNSUPPORTED;
  int rc = make_tma_blocks(&p.tmA, a.A, a.M, a.K, kCols, p.copy);
  if (rc == EPILORA_OK) rc = make_tma_blocks(&p.tmB, a.W, w_rows, a.K, kTileN, p.copy);
  if (rc != EPILORA_OK) return rc;
  const int sms = num_sms();
  p.splits = kGrouped ? 1 : few_splits(a.N, a.K);
  const int extra = 1024 + kMisc + kSumBytes<kGated> + (kGrouped ? 2 * (p.experts + 1) * 4 : 0);
  const int stage = p.copy * ((kGated ? 2 : 1) * kWBytes + kABytes);
  p.stages = (227 * 1024 - extra) / stage;
  if (p.stages > kStagesMax) p.stages = kStagesMax;
  const int smem = p.stages * stage + extra;
  const auto kern = block_few_kernel<kGated>;
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EPILORA_ERR_CUDA;
  if (attr_done[dev] < smem) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
      return EPILORA_ERR_CUDA;
    attr_done[dev] = 227 * 1024;
  }
  // (split: a tile per cluster; few rows are one tile of them)
  const unsigned grid = kGrouped ? sms : p.splits * p.n_tiles;
  return launch_dependent(kern, grid, kThreads, smem, a.stream, p, p.splits);
}

}  // namespace

// The product turned round pays where the sums are gated (up projections of 1, 8 and 64 tokens 35.6 -> 29.1, 99 -> 78
// and 153 -> 132 us), and where K is split (32 x 14336 -> 4096: 29.7 -> 18.5 us). Otherwise block_gemm.cu's narrower
// tiles spread better over the SMs (32 x 4096 -> 28672: 26.4 against 30.6 us; down projections of 64 tokens 88 against
// 99). The host knows the mean of an expert's rows alone: where all tokens go to the same few experts their weights are
// read again for every 32 rows (128 tokens with the same eight experts, or with one: 52 us).
bool block_few_takes(const BlockGemmArgs& a) {
  if (a.grouped) return a.gated && a.M / a.experts <= kCols / 2;
  return a.M <= kCols && few_splits(a.N, a.K) > 1;
}

int launch_block_few(const BlockGemmArgs& a) { return a.gated ? launch<true>(a) : launch<false>(a); }

}  // namespace epi
