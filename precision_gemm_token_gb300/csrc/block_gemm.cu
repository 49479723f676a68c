// Product of block-quantized rows with block-scaled weights, on tcgen05
// (kind::f8f6f4, E4M3 x E4M3), for plain matrices and for the experts of a
// mixture (the rows of an expert times that expert's weights).
//
//   y[m][n] = sum_b as[b][m] ws[n / 128][b] sum_{k in block b} A[m][k] W[n][k]
//
// A scale holds for 128 elements of K, so the tensor core's accumulator is
// good for one block only: four MMAs (K = 32 each) put a block's products in
// TMEM, the summing warps read them and add them, times the two scales, to
// fp32 sums in registers. TMEM is two halves of 256 columns, filled and read
// in turn; a half holds a group of 256 / BN blocks, so that a narrow tile's
// warps wait as rarely, and have as many loads under way, as a wide one's.
//
// Roles (384 threads, one CTA per SM, walking its tiles of 128 rows x BN
// columns):
//   warp 0       TMA copies of A and W, a block a stage of the ring
//   warp 1       MMA issue
//   warps 2, 3   the scales of the groups to come, into a ring of their own
//                (each block needs new ones: the summing warps would wait for
//                memory at every block)
//   warps 4..11  sums: each warp 32 rows (its TMEM lanes) by half the columns,
//                a thread one row; then the scales are one factor per thread
//                and block, and a row's output needs no exchange
// Gated products take 128 columns of gate and the same 128 of up as one tile,
// so that a thread holds both of an element and two threads a whole block of
// the output, which leaves quantized.
//
// Bound: the loop between the MMAs and the sums. 2048 x 8192 -> 28672 takes 396 us (437 us after seconds of it, at the
// clock that the power limit leaves), 2.4 (2.2) PFLOP/s, 62 (56) % of twice the measured bf16 rate: 980 cycles a block
// of 128 x 256, where the MMAs take 512 and the 96 KB that go through shared memory some 820; without the sums a block
// takes 850. Down projections of 64 tokens over 64 experts of 4096 x 1792 read their 470 MB at 6.3 TB/s.
//
// Every wait is bounded: on a timeout the CTA records EPILORA_ERR_TIMEOUT,
// stops issuing, waits (bounded) for its copies and MMAs in flight, writes NaN
// for the sums that are not whole and frees its TMEM.
#include "block_gemm.cuh"

namespace epi {

namespace {

constexpr int kRows = 128;                     // rows of a tile (TMEM lanes)
constexpr int kThreads = 384;
constexpr int kSumThreads = 256;
constexpr int kABytes = kRows * kBlock;        // a stage's rows of A
constexpr int kSumBarrier = 1;
// registers: 168 a thread at launch (64,512); the sums' warps take what the others give back
constexpr int kRegsOther = 40, kRegsSum = 232;
constexpr int kHalf = 256;                     // columns of a half of TMEM
constexpr int kScaleBlocks = 32;               // blocks in the scales' ring
constexpr int kTurnedRow = 9;                  // words of a staged row of 16 outputs
constexpr int kScaleRow = kRows + 4;           // a block's scales: of the rows, then up to two of the weights

template <int BN>
struct Cfg {
  static constexpr int kBBytes = BN * kBlock;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kGroup = kHalf / BN;    // blocks of a group
  static constexpr int kStagesMax = 16;
  static constexpr int kSlots = kScaleBlocks / kGroup;       // groups in the scales' ring
  // barriers, amax exchange, scales
  static constexpr int kMisc = 1024 + 2 * 2 * kRows * 4 + kScaleBlocks * kScaleRow * 4;
};

struct Params {
  CUtensorMap tmA, tmB;
  const float* a_scale;
  const float* w_scale;
  int64_t a_scale_ld, ldy;
  void* Y;
  uint8_t* inner;
  float* inner_scale;
  const int32_t* offsets;      // grouped: rows of expert e are [offsets[e], offsets[e + 1])
  const int32_t* out_rows;     // the output row of each row (NULL: the same)
  int* status;
  int M, N, kb;
  int n_tiles, experts;
  int stages, wide_store, early_weights;
  int late;                    // the test hook: the block whose copies never seem complete, else -1
};

__device__ __forceinline__ void sums_barrier() {
  asm volatile("bar.sync %0, %1;" ::"n"(kSumBarrier), "n"(kSumThreads) : "memory");
}

// acc += x * f for a register of a TMEM load: volatile, so that it stays behind the wait for the load. One
// multiply-add at a time: those of two need their operands in pairs of registers, which costs a move each.
__device__ __forceinline__ void fma_loaded(float& acc, uint32_t x, float f) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(x)), "f"(f));
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N]) {
  if constexpr (N == 16)
    tmem_ld_32x32b_x16(taddr, v);
  else
    tmem_ld_32x32b_x32(taddr, v);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// kF32: grouped products that leave in fp32, 512 bytes a thread instead of 256 (down projections of 4096 tokens, sum
// and all, 536 us instead of 380, of 64 tokens 89.4 instead of 83.3, of one 23.2 instead of 22.2: the parts' traffic)
template <int BN, bool kGrouped, bool kGated, bool kF32>
__global__ void __launch_bounds__(kThreads, 1) block_gemm_kernel(const __grid_constant__ Params p) {
  using C = Cfg<BN>;
  constexpr int NC = BN / 2;                    // columns of a summing thread
  constexpr int CH = NC < 32 ? NC : 32;         // of them per TMEM load
  constexpr int LOADS = 64 / CH;                // loads under way together (some 200 cycles each, whatever the size)
  constexpr int G = C::kGroup;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stages = p.stages, kb = p.kb;
  uint8_t* misc = smem + static_cast<size_t>(stages) * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + C::kStagesMax;
  uint64_t* filled = empty + C::kStagesMax;     // [2] a half holds a group's products, and the ring its scales
  uint64_t* drained = filled + 2;               // [2] they have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* amax = reinterpret_cast<float*>(misc + 1024);                 // [2][2][kRows]
  float* scales = amax + 4 * kRows;                                    // [kScaleBlocks][kScaleRow]
  uint32_t* staged = reinterpret_cast<uint32_t*>(misc + C::kMisc);      // [8 warps][32][kTurnedRow], plain only
  int* offsets = reinterpret_cast<int*>(misc + C::kMisc);              // [experts + 1], grouped only
  int* starts = offsets + p.experts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&filled[b], 3);                 // the products, and the two scale warps
      mbar_init(&drained[b], kSumThreads / 32);
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
    // row tiles before each expert: one warp, 32 experts at a time
    pdl_wait_primary();
    if (warp == 2) fill_walk<kRows>(p.offsets, p.experts, offsets, starts, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_allow_dependents();
  const uint32_t tmem_base = *tmem_slot;
  Walk<kGrouped, kRows> walk(p.M, p.n_tiles, p.experts, offsets, starts);

  // The sums' wait of a wide tile polls, with as little code as can be: a warp that the hardware suspended wakes some
  // 100 cycles late, which is 3 % of a call with many rows (and 2 % lost on narrow tiles, whose warps mostly do wait).
  // Gives up after 10^7 polls.
  const auto poll = [&](uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    for (int i = 0; i < 10000000; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(at), "r"(parity)
          : "memory");
      if (ok != 0) return true;
    }
    return false;
  };
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
        for (int t = blockIdx.x; t < walk.total && go; t += gridDim.x) {
          const Tile tile = walk.at(t);
          const int n0 = tile.n * (kGated ? kBlock : BN);
          const int wrow = tile.expert * (kGated ? 2 : 1) * p.N + n0;
          const auto copy_w = [&](int st, int b) {
            uint8_t* dst = smem + static_cast<size_t>(st) * C::kStage + kABytes;
            mbar_arrive_expect_tx(&full[st], C::kStage + (b == p.late ? 16 : 0));
            tma_load_2d(dst, &p.tmB, &full[st], b * kBlock, wrow);
            if (kGated) tma_load_2d(dst + kBlock * kBlock, &p.tmB, &full[st], b * kBlock, wrow + p.N);
          };
          // the first tile of a plain product: weights of the first stages before the rows are there
          int early = 0;
          if (!waited) {
            early = p.early_weights ? min(stages, kb) : 0;
            for (int b = 0; b < early; ++b) copy_w(b, b);
            issued |= (1u << early) - 1u;
            pdl_wait_primary();
            fence_proxy_async_global();
            waited = true;
          }
          for (int b = 0; b < kb; ++b) {
            if (!wait(&empty[s], ph ^ 1u)) {
              go = false;
              break;
            }
            if (b >= early) copy_w(s, b);
            tma_load_2d(smem + static_cast<size_t>(s) * C::kStage, &p.tmA, &full[s], b * kBlock, tile.first);
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
        constexpr uint32_t kIdesc = idesc_f8f6f4_e4m3(kRows, BN);
        const uint64_t desc0 = make_smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        int s = 0, half = 0;
        uint32_t ph = 0, hph = 0;
        bool go = true, any = false;
        for (int t = blockIdx.x; t < walk.total && go; t += gridDim.x) {
          for (int b0 = 0; b0 < kb; b0 += G) {
            if (!wait(&drained[half], hph ^ 1u)) {
              go = false;
              break;
            }
            const int n = min(G, kb - b0);
            for (int u = 0; u < n; ++u) {
              if (!wait(&full[s], ph)) {
                go = false;
                break;
              }
              tc_fence_after();
              // (descriptors count 16 bytes: 2 more for each 32 bytes of K)
              const uint64_t ad = desc0 + s * (C::kStage >> 4), bd = ad + (kABytes >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f8f6f4(tmem_base + half * kHalf + u * BN, ad + 2 * kk, bd + 2 * kk, kIdesc, kk > 0);
              tc_commit(&empty[s]);
              any = true;
              if (++s == stages) {
                s = 0;
                ph ^= 1u;
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
    } else {
      // ===== scales =====
      constexpr int kAhead = C::kSlots - 2;     // groups under way (the slot before the last one may be read still)
      const int i = static_cast<int>(threadIdx.x) - 64;
      const int nb = n_blocks(p.N);
      constexpr int kW = BN == 256 ? 2 : 1;     // scales of the weights per block
      pdl_wait_primary();
      Walk<kGrouped, kRows> ahead = walk;
      int c_t = blockIdx.x, c_b = 0, put = 0;
      Tile tile{};
      const float *c_a = nullptr, *c_w = nullptr;
      const auto enter = [&] {
        tile = ahead.at(c_t);
        c_a = p.a_scale + tile.first;
        const int w = i % kW;                   // (threads below kW * G)
        const int block = kGated ? (tile.expert * 2 + w) * nb + tile.n
                                 : tile.expert * nb + min(tile.n * BN / kBlock + w, nb - 1);
        c_w = p.w_scale + static_cast<int64_t>(block) * kb;
      };
      const auto fetch = [&] {
        if (c_t < ahead.total) {
          float* slot = scales + put * (G * kScaleRow);
          const int n = min(G, kb - c_b);
          for (int u = 0; u < n; ++u) {
            const float* src = c_a + (c_b + u) * p.a_scale_ld;
            if (i < tile.rows) copy4(slot + u * kScaleRow + i, src + i);
            if (i + 64 < tile.rows) copy4(slot + u * kScaleRow + i + 64, src + i + 64);
          }
          if (i < kW * n) copy4(slot + (i / kW) * kScaleRow + kRows + i % kW, c_w + c_b + i / kW);
          put = (put + 1) & (C::kSlots - 1);
          c_b += G;
          if (c_b >= kb) {
            c_b = 0;
            c_t += gridDim.x;
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
      for (int t = blockIdx.x; t < walk.total && go; t += gridDim.x)
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
  } else {
    // ===== sums =====
    setmaxnreg_inc<kRegsSum>();
    pdl_wait_primary();
    const int side = (warp - 4) >> 2;           // of the columns
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int half = 0, turn = 0, take = 0;
    uint32_t hph = 0;
    bool dead = false;
    for (int t = blockIdx.x; t < walk.total; t += gridDim.x, turn ^= 1) {
      const Tile tile = walk.at(t);
      const bool live = r < tile.rows;
      const bool warp_live = (warp & 3) * 32 < tile.rows;
      const int row = tile.first + (live ? r : 0);
      const int slot = p.out_rows != nullptr ? __ldcg(p.out_rows + row) : row;
      // this side's first column
      const int n0 = kGated ? tile.n * kBlock + side * (NC / 2) : tile.n * BN + side * NC;
      const bool cols = n0 < p.N;
      const float start = dead ? __int_as_float(0x7fffffff) : 0.0f;
      float acc[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) acc[i] = start;
#pragma unroll 1
      for (int b0 = 0; b0 < kb; b0 += G) {
        if (!dead && !__all_sync(0xffffffffu, BN == 256 ? poll(&filled[half], hph) : wait(&filled[half], hph)))
          dead = true;
        if (!dead) {
          tc_fence_after();
          const auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&drained[half]);
          };
          if (warp_live) {
            const int n = min(G, kb - b0);
            const float* sc = scales + take * (G * kScaleRow);
            // piece c of the 128 columns that a thread has in a half: block c * CH / NC of the group, from column
            // c * CH % NC of the thread's; gated: its first half gate, its second up
            const auto at = [&](int c) {
              const int u = c * CH / NC, col = c * CH % NC;
              return lanes + half * kHalf + u * BN +
                     (kGated ? (col >= NC / 2 ? kBlock + col - NC / 2 : col) + side * (NC / 2) : side * NC + col);
            };
            const auto block = [&](int c) { return c * CH / NC; };
            const auto there = [&](int c) { return block(c) == 0 || block(c) < n; };
            const auto column = [&](int c) { return c * CH % NC; };
            const auto factor = [&](int c) {
              const int w = kGated ? column(c) >= NC / 2 : BN == 256 ? side : 0;
              return sc[block(c) * kScaleRow + r] * sc[block(c) * kScaleRow + kRows + w];
            };
            const auto add = [&](int c, uint32_t (&x)[CH], float f) {
#pragma unroll
              for (int i = 0; i < CH; ++i) fma_loaded(acc[column(c) + i], x[i], f);
            };
            uint32_t v[LOADS][CH];
            float f[LOADS];
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
              if (there(i)) tmem_ld(at(i), v[i]);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) f[i] = factor(i);
            tmem_ld_wait();
            const bool more = there(LOADS);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
              if (there(i)) add(i, v[i], f[i]);
              if (there(LOADS + i)) tmem_ld(at(LOADS + i), v[i]);
            }
#pragma unroll
            for (int i = 0; i < LOADS; ++i) f[i] = factor(LOADS + i);
            tmem_ld_wait();
            // the half and its scales are in registers: the next group may have both
            release();
            if (more) {
#pragma unroll
              for (int i = 0; i < LOADS; ++i)
                if (there(LOADS + i)) add(LOADS + i, v[i], f[i]);
            }
          } else {
            release();
          }
        }
        take = (take + 1) & (C::kSlots - 1);
        half ^= 1;
        if (half == 0) hph ^= 1u;
      }
      if (dead && start == 0.0f) {              // sums that are not whole: the tile once more, as NaN
        t -= static_cast<int>(gridDim.x);
        turn ^= 1;
        continue;
      }
      if constexpr (kGated) {
        constexpr int H = NC / 2;              // elements of the output per thread
        float h[H], m = 0.0f;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          h[i] = n0 + i < p.N ? silu(acc[i]) * acc[H + i] : 0.0f;
          m = fmaxf(m, fabsf(h[i]));
        }
        amax[(turn * 2 + side) * kRows + r] = m;
        sums_barrier();
        m = fmaxf(m, amax[(turn * 2 + (side ^ 1)) * kRows + r]);
        const float s = block_scale(m);
        const BlockDiv by = block_div(s);
        if (live) {
          uint8_t* out = p.inner + static_cast<int64_t>(slot) * p.N + n0;
#pragma unroll
          for (int c = 0; c < H; c += 16) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float d[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) d[e] = div_rn_by_recip(h[c + 4 * i + e], by.s, by.rs);
              q[i] = cvt_e4m3x2(d[0], d[1]) | (cvt_e4m3x2(d[2], d[3]) << 16);
            }
            if (n0 + c < p.N) *reinterpret_cast<uint4*>(out + c) = make_uint4(q[0], q[1], q[2], q[3]);
          }
          if (side == 0) p.inner_scale[static_cast<int64_t>(tile.n) * p.M + slot] = s;
        }
      } else if constexpr (kF32) {
        if (live) {
          float* const Y = static_cast<float*>(p.Y) + slot * p.ldy + n0;
#pragma unroll
          for (int c = 0; c < NC; c += 8) {
            uint32_t q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __float_as_uint(acc[c + i]);
            if (n0 + c < p.N) st_global_v8(Y + c, q);
          }
        }
      } else if (warp_live && cols) {
        __nv_bfloat16* const Y = static_cast<__nv_bfloat16*>(p.Y);
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          uint32_t q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = pack_bf16x2(acc[c + 2 * i], acc[c + 2 * i + 1]);
          if (kGrouped || (p.wide_store && n0 + c + 16 <= p.N)) {
            if (live && (!kGrouped || n0 + c < p.N)) st_global_v8(Y + slot * p.ldy + n0 + c, q);
          } else {
            // rows that start anywhere, and the last columns: turned round in shared memory, two rows of 16 a store (a
            // thread's own row element by element would touch 32 sectors a store)
            uint32_t* const turned = staged + (warp - 4) * 32 * kTurnedRow;
#pragma unroll
            for (int i = 0; i < 8; ++i) turned[lane * kTurnedRow + i] = q[i];
            __syncwarp();
            const int n = n0 + c + (lane & 15);
#pragma unroll 4
            for (int i = lane >> 4; i < 32; i += 2)
              if ((warp & 3) * 32 + i < tile.rows && n < p.N)
                reinterpret_cast<uint16_t*>(Y)[(tile.first + (warp & 3) * 32 + i) * p.ldy + n] =
                    reinterpret_cast<const uint16_t*>(turned + i * kTurnedRow)[lane & 15];
            __syncwarp();
          }
        }
      }
    }
    if (dead) {
      *abort_flag = 1;
      record_status(p.status, EPILORA_ERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kHalf);
  }
}

template <int BN, bool kGrouped, bool kGated, bool kF32 = false>
int launch(const BlockGemmArgs& a) {
  using C = Cfg<BN>;
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
  p.late = block_test_late_copies() ? p.kb - 1 : -1;
  const int width = kGated ? kBlock : BN;
  p.n_tiles = (a.N + width - 1) / width;
  p.wide_store = (reinterpret_cast<uintptr_t>(a.Y) & 31) == 0 && a.ldy % 16 == 0;
  const int64_t w_rows = static_cast<int64_t>(p.experts) * a.N * (kGated ? 2 : 1);
  // tiles, and rows of the tensor maps, are counted in 31 bits
  const int64_t tiles = (static_cast<int64_t>(a.M) / kRows + 1 + (kGrouped ? p.experts : 0)) * p.n_tiles;
  if (tiles > EPILORA_BLOCK_MAX_SIZE || w_rows > EPILORA_BLOCK_MAX_SIZE) return EPILORA_ERR_UNSUPPORTED;
  int rc = make_tma_2d_u8(&p.tmA, a.A, a.M, a.K, a.K, kRows, kBlock, true);
  if (rc == EPILORA_OK) rc = make_tma_2d_u8(&p.tmB, a.W, w_rows, a.K, a.K, kGated ? kRows : BN, kBlock, true);
  if (rc != EPILORA_OK) return rc;
  const int extra = 1024 + C::kMisc + (kGrouped ? 2 * (p.experts + 1) * 4 : kSumThreads * kTurnedRow * 4);
  p.stages = (227 * 1024 - extra) / C::kStage;
  if (p.stages > C::kStagesMax) p.stages = C::kStagesMax;
  const int smem = p.stages * C::kStage + extra;
  const auto kern = block_gemm_kernel<BN, kGrouped, kGated, kF32>;
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EPILORA_ERR_CUDA;
  if (attr_done[dev] < smem) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
      return EPILORA_ERR_CUDA;
    attr_done[dev] = 227 * 1024;
  }
  const int sms = num_sms();
  const unsigned grid = kGrouped || tiles > sms ? sms : static_cast<unsigned>(((a.M + kRows - 1) / kRows) * p.n_tiles);
  return launch_dependent(kern, grid < 1 ? 1 : grid, kThreads, smem, a.stream, p);
}

}  // namespace

// Tiles of BN columns: as wide as pays. A block of K costs a CTA 0.50, 0.31, 0.21 or 0.20 us at 256, 128, 64 and 32
// columns; a call takes as many of them as its fullest CTA has tiles (one token, 4096 -> 6144: 20.7, 14.4, 11.5 and
// 17.6 us; 509 tokens, 2064 -> 1000, with ends 4 us longer than now: 46, 28, 18 and 15; 2048 tokens, 8192 -> 28672:
// 395, 568, 854 and 1416).
static int tile_width(int M, int N) {
  const int widths[4] = {256, 128, 64, 32}, costs[4] = {50, 31, 21, 20};
  const int64_t sms = num_sms(), mt = (M + kRows - 1) / kRows;
  int best = 256;
  int64_t least = 0;
  for (int i = 0; i < 4; ++i) {
    const int64_t cost = (mt * ((N + widths[i] - 1) / widths[i]) + sms - 1) / sms * costs[i];
    if (i == 0 || cost < least) best = widths[i], least = cost;
  }
  return best;
}

int launch_block_gemm(const BlockGemmArgs& a) {
  if (block_few_takes(a)) return launch_block_few(a);
  if (a.gated) return launch<256, true, true>(a);
  if (a.grouped) return a.f32 ? launch<256, true, false, true>(a) : launch<256, true, false>(a);
  switch (tile_width(a.M, a.N)) {
    case 256: return launch<256, false, false>(a);
    case 128: return launch<128, false, false>(a);
    case 64: return launch<64, false, false>(a);
    default: return launch<32, false, false>(a);
  }
}

}  // namespace epi
