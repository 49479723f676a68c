// Product of block-quantized rows with block-scaled weights, on tcgen05
// (kind::f8f6f4, E4M3 x E4M3), for plain matrices and for the experts of a
// mixture (the rows of an expert times that expert's weights).
//
//   y[m][n] = sum_b as[b][m] ws[n / 128][b] sum_{k in block b} A[m][k] W[n][k]
//
// A scale holds for 128 elements of K, so the tensor core's accumulator is
// good for one block only: four MMAs (K = 32 each) fill a TMEM buffer with a
// block's products, the accumulating warps read it and add it, times the two
// scales, to fp32 sums in registers while the next buffer fills.
//
// Roles (384 threads, one CTA per SM, walking its tiles of 128 rows x BN
// columns):
//   warp 0       copies: rows of A (one box, or four rows a gather for the
//                rows of an expert) and of W through a ring of 128-byte stages
//   warp 1       MMA issue
//   warps 4..11  sums: each warp 32 rows (its TMEM lanes) by half the columns,
//                a thread one row; then the scales are one factor per thread
//                and block, and a row's output needs no exchange
// Gated products take 128 columns of gate and the same 128 of up as one tile,
// so that a thread holds both of an element and two threads a whole block of
// the output, which leaves quantized.
//
// Every wait is bounded: on a timeout the CTA records EPILORA_ERR_TIMEOUT,
// stops issuing, waits (bounded) for its copies and MMAs in flight and frees
// its TMEM.
#include "block_quant.cuh"

namespace epi {

namespace {

constexpr int kRows = 128;                     // rows of a tile (TMEM lanes)
constexpr int kThreads = 384;
constexpr int kSumThreads = 256;
constexpr int kABytes = kRows * kBlock;        // a stage's rows of A
constexpr int kSumBarrier = 1;
// registers: 168 a thread at launch (64,512); the sums' warps take what the others give back
constexpr int kRegsOther = 40, kRegsSum = 232;

template <int BN>
struct Cfg {
  static constexpr int kBBytes = BN * kBlock;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kBufs = BN >= 256 ? 2 : 4;
  static constexpr int kTmemCols = kBufs * BN;
  static constexpr int kStagesMax = 10;
  static constexpr int kMisc = 2048 + 2 * 2 * kRows * 4;     // barriers, amax exchange
};

struct Params {
  CUtensorMap tmA, tmB;
  const float* a_scale;
  const float* w_scale;
  int64_t a_scale_ld, ldy;
  void* Y;
  uint8_t* inner;
  float* inner_scale;
  MoePlan plan;
  int* status;
  int M, N, K, kb;
  int n_tiles, experts, slot_div;
  int stages, wide_store, early_weights;
};

struct Tile {
  int expert, first, rows, n;      // rows [first, first + rows) of the expert's list, columns' tile
};

// The tiles of a CTA in order: expert by expert, its row tiles fastest (CTAs
// next to one another then share weights in L2).
template <bool kGrouped>
struct Walk {
  const int* offsets;        // shared memory: [experts + 1]
  const int* starts;         // row tiles before each expert, [experts + 1]
  int n_tiles, M, e, total;
  __device__ Walk(const Params& p, const int* off, const int* st) : offsets(off), starts(st), n_tiles(p.n_tiles), M(p.M), e(0) {
    total = (kGrouped ? starts[p.experts] : (p.M + kRows - 1) / kRows) * n_tiles;
  }
  __device__ Tile at(int t) {
    Tile r;
    if (kGrouped) {
      while (starts[e + 1] * n_tiles <= t) ++e;
      const int mt = starts[e + 1] - starts[e], local = t - starts[e] * n_tiles;
      const int m = local % mt;
      r.expert = e;
      r.n = local / mt;
      r.first = offsets[e] + m * kRows;
      r.rows = min(kRows, offsets[e + 1] - r.first);
    } else {
      const int mt = total / n_tiles, m = t % mt;
      r.expert = 0;
      r.n = t / mt;
      r.first = m * kRows;
      r.rows = min(kRows, M - r.first);
    }
    return r;
  }
};

// Four rows of a 2D tensor map (box one row high), 128 bytes each from column x (a multiple of 128).
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int4 rows) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(rows.x), "r"(rows.y),
      "r"(rows.z), "r"(rows.w)
      : "memory");
}

__device__ __forceinline__ void sums_barrier() { asm volatile("bar.sync %0, %1;" ::"n"(kSumBarrier), "n"(kSumThreads) : "memory"); }

template <int N>
__device__ __forceinline__ void loaded(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
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

template <int BN, bool kGrouped, bool kGated>
__global__ void __launch_bounds__(kThreads, 1) block_gemm_kernel(const __grid_constant__ Params p) {
  using C = Cfg<BN>;
  constexpr int NC = BN / 2;                    // columns of a summing thread
  constexpr int CH = NC < 32 ? NC : 32;         // of them per TMEM load
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stages = p.stages, kb = p.kb;
  uint8_t* misc = smem + static_cast<size_t>(stages) * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + C::kStagesMax;
  uint64_t* filled = empty + C::kStagesMax;     // [kBufs] a block's products are in the buffer
  uint64_t* drained = filled + C::kBufs;        // [kBufs] they have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + C::kBufs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* amax = reinterpret_cast<float*>(misc + 2048);                 // [2][2][kRows]
  int* offsets = reinterpret_cast<int*>(misc + C::kMisc);              // [experts + 1], grouped only
  int* starts = offsets + p.experts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&filled[b], 1);
      mbar_init(&drained[b], kSumThreads / 32);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (kGrouped) {
    // row tiles before each expert: one warp, 32 experts at a time
    pdl_wait_primary();
    if (warp == 2) {
      int before = 0;
      for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int e = e0 + lane;
        const int o0 = e <= p.experts ? __ldcg(p.plan.offsets + e) : 0;
        const int o1 = e < p.experts ? __ldcg(p.plan.offsets + e + 1) : o0;
        const int mt = (o1 - o0 + kRows - 1) / kRows;
        int sum = mt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        if (e < p.experts) {
          offsets[e] = o0;
          starts[e] = before + sum - mt;
          if (e == p.experts - 1) {
            offsets[e + 1] = o1;
            starts[e + 1] = before + sum;
          }
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_allow_dependents();
  const uint32_t tmem_base = *tmem_slot;
  Walk<kGrouped> walk(p, offsets, starts);

  // gives up when the wait runs out or another role has
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag == 0 && mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
    if (*abort_flag == 0) {
      *abort_flag = 1;
      record_status(p.status, EPILORA_ERR_TIMEOUT);
    }
    return false;
  };

  if (warp < 4) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == 0) {
      // ===== copies =====
      int s = 0;
      uint32_t ph = 0, issued = 0, phases = 0;
      bool go = true, waited = kGrouped;
      for (int t = blockIdx.x; t < walk.total && go; t += gridDim.x) {
        const Tile tile = walk.at(t);
        const int n0 = tile.n * (kGated ? kBlock : BN);
        const int wrow = kGated ? tile.expert * 2 * p.N + n0 : tile.expert * p.N + n0;
        int4 arow = make_int4(0, 0, 0, 0);
        if (kGrouped) {
          // this lane's four rows; behind the last row, the last row again
          int v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = __ldcg(p.plan.rows + tile.first + min(4 * lane + i, tile.rows - 1)) / p.slot_div;
          arow = make_int4(v[0], v[1], v[2], v[3]);
        }
        const int gathers = (tile.rows + 3) / 4;
        const uint32_t bytes = C::kBBytes + (kGrouped ? gathers * 4 * kBlock : kABytes);
        const auto copy_b = [&](int st, int b) {
          uint8_t* dst = smem + static_cast<size_t>(st) * C::kStage + kABytes;
          tma_load_2d(dst, &p.tmB, &full[st], b * kBlock, wrow);
          if (kGated) tma_load_2d(dst + kABytes, &p.tmB, &full[st], b * kBlock, wrow + p.N);
        };
        // the first tile of a plain product: weights of the first stages before the rows are there
        const int early = !waited && p.early_weights ? min(stages, kb) : 0;
        if (!kGrouped && !waited) {
          if (lane == 0)
            for (int b = 0; b < early; ++b) {
              mbar_arrive_expect_tx(&full[b], bytes);
              copy_b(b, b);
            }
          pdl_wait_primary();
          fence_proxy_async_global();
          waited = true;
          issued |= (1u << early) - 1u;
        }
        if (kGrouped) fence_proxy_async_global();
        for (int b = 0; b < kb; ++b) {
          if (!wait(&empty[s], ph ^ 1u)) go = false;
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          uint8_t* dst = smem + static_cast<size_t>(s) * C::kStage;
          if (lane == 0 && b >= early) {
            mbar_arrive_expect_tx(&full[s], bytes);
            copy_b(s, b);
          }
          if (kGrouped) {
            __syncwarp();
            if (lane < gathers) tma_gather4(dst + lane * 4 * kBlock, &p.tmA, &full[s], b * kBlock, arow);
          } else if (lane == 0) {
            tma_load_2d(dst, &p.tmA, &full[s], b * kBlock, tile.first);
          }
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
    } else if (warp == 1) {
      // ===== MMA issue =====
      if (elect_one()) {
        constexpr uint32_t kIdesc = idesc_f8f6f4_e4m3(kRows, BN);
        int s = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        bool go = true, any = false;
        int last = 0;
        uint32_t last_ph = 0;
        for (int t = blockIdx.x; t < walk.total && go; t += gridDim.x) {
          for (int b = 0; b < kb; ++b) {
            if (!wait(&drained[buf], bph ^ 1u) || !wait(&full[s], ph)) {
              go = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_at = smem_u32(smem + static_cast<size_t>(s) * C::kStage), b_at = a_at + kABytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8f6f4(tmem_base + buf * BN, make_smem_desc(a_at + kk * 32, 16, 1024, kSwizzle128B),
                         make_smem_desc(b_at + kk * 32, 16, 1024, kSwizzle128B), kIdesc, kk > 0);
            tc_commit(&empty[s]);
            tc_commit(&filled[buf]);
            any = true;
            last = buf;
            last_ph = bph;
            if (++s == stages) {
              s = 0;
              ph ^= 1u;
            }
            if (++buf == C::kBufs) {
              buf = 0;
              bph ^= 1u;
            }
          }
        }
        // nothing of this thread in flight at exit: the last commit covers every MMA before it
        if (any) (void)mbar_wait_bounded(&filled[last], last_ph, kWaitLimitNs);
      }
      __syncwarp();
    }
  } else {
    // ===== sums =====
    setmaxnreg_inc<kRegsSum>();
    pdl_wait_primary();
    const int half = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int buf = 0, turn = 0;
    uint32_t bph = 0;
    bool dead = false;
    for (int t = blockIdx.x; t < walk.total; t += gridDim.x, turn ^= 1) {
      const Tile tile = walk.at(t);
      const bool live = r < tile.rows;
      const bool warp_live = (warp & 3) * 32 < tile.rows;
      const int slot = !live ? 0 : kGrouped ? __ldcg(p.plan.rows + tile.first + r) : tile.first + r;
      const float* as = p.a_scale + (kGrouped ? slot / p.slot_div : slot);
      // this half's first column, and the rows of scales that its columns have
      const int n0 = kGated ? tile.n * kBlock + half * NC / 2 : tile.n * BN + half * NC;
      const int nb = n_blocks(p.N);
      const int wb = kGated ? tile.expert * 2 * nb + tile.n : tile.expert * nb + n0 / kBlock;
      const bool cols = n0 < p.N;
      const float* ws = p.w_scale + static_cast<int64_t>(cols ? wb : 0) * kb;
      uint64_t acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
      float as_next = __ldcg(as), w0_next = __ldcg(ws), w1_next = kGated ? __ldcg(ws + static_cast<int64_t>(nb) * kb) : 0.0f;
      for (int b = 0; b < kb; ++b) {
        const float f0 = as_next * w0_next, f1 = as_next * w1_next;
        if (b + 1 < kb) {
          as_next = __ldcg(as + (b + 1) * p.a_scale_ld);
          w0_next = __ldcg(ws + b + 1);
          if (kGated) w1_next = __ldcg(ws + static_cast<int64_t>(nb) * kb + b + 1);
        }
        if (!dead && !__all_sync(0xffffffffu, wait(&filled[buf], bph))) dead = true;
        if (!dead) {
          tc_fence_after();
          if (warp_live) {
            // gated: the first half of the registers gate, the second up
            const auto at = [&](int c) {
              return lanes + buf * BN + (kGated ? (c >= NC / 2 ? kBlock + c - NC / 2 : c) + half * (NC / 2) : half * NC + c);
            };
            uint32_t v[2][CH];
            tmem_ld(at(0), v[0]);
#pragma unroll
            for (int c = 0; c < NC; c += CH) {
              uint32_t (&x)[CH] = v[(c / CH) & 1];
              tmem_ld_wait();
              loaded(x);
              if (c + CH < NC) tmem_ld(at(c + CH), v[(c / CH + 1) & 1]);
              const float f = kGated && c >= NC / 2 ? f1 : f0;
              const uint64_t ff = f32x2(f, f);
#pragma unroll
              for (int i = 0; i < CH / 2; ++i)
                acc[c / 2 + i] = fma_f32x2(f32x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), ff, acc[c / 2 + i]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&drained[buf]);
        }
        if (++buf == C::kBufs) {
          buf = 0;
          bph ^= 1u;
        }
      }
      if constexpr (kGated) {
        constexpr int H = NC / 2;              // elements of the output per thread
        float h[H], m = 0.0f;
#pragma unroll
        for (int i = 0; i < H; i += 2) {
          float g[2], u[2];
          f32x2_parts(acc[i / 2], g[0], g[1]);
          f32x2_parts(acc[H / 2 + i / 2], u[0], u[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            h[i + q] = n0 + i + q < p.N ? __fdiv_rn(g[q], 1.0f + expf(-g[q])) * u[q] : 0.0f;
            m = fmaxf(m, fabsf(h[i + q]));
          }
        }
        float* mine = amax + (turn * 2 + half) * kRows;
        mine[r] = m;
        sums_barrier();
        m = fmaxf(m, amax[(turn * 2 + (half ^ 1)) * kRows + r]);
        const float s = block_scale(m), rs = __fdiv_rn(1.0f, s);
        const bool plain = block_scale_plain(s);
        if (live && !dead) {
          uint8_t* out = p.inner + static_cast<int64_t>(slot) * p.N + n0;
#pragma unroll
          for (int c = 0; c < H; c += 16) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float d[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) d[e] = plain ? div_rn_by_recip(h[c + 4 * i + e], s, rs) : __fdiv_rn(h[c + 4 * i + e], s);
              q[i] = cvt_e4m3x2(d[0], d[1]) | (cvt_e4m3x2(d[2], d[3]) << 16);
            }
            if (n0 + c < p.N) *reinterpret_cast<uint4*>(out + c) = make_uint4(q[0], q[1], q[2], q[3]);
          }
          if (half == 0) p.inner_scale[static_cast<int64_t>(tile.n) * p.M + slot] = s;
        }
      } else if (live && cols && !dead) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.Y) + slot * p.ldy + n0;
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          uint32_t q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float lo, hi;
            f32x2_parts(acc[c / 2 + i], lo, hi);
            q[i] = pack_bf16x2(lo, hi);
          }
          if (p.wide_store && n0 + c + 16 <= p.N) {
            st_global_v8(out + c, q);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (n0 + c + i < p.N) reinterpret_cast<uint16_t*>(out)[c + i] = static_cast<uint16_t>(q[i / 2] >> (16 * (i & 1)));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int BN, bool kGrouped, bool kGated>
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
  p.plan = a.plan;
  p.status = a.status;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.kb = n_blocks(a.K);
  p.experts = kGrouped ? a.experts : 1;
  p.slot_div = a.slot_div;
  p.early_weights = a.early_weights;
  const int width = kGated ? kBlock : BN;
  p.n_tiles = (a.N + width - 1) / width;
  p.wide_store = (reinterpret_cast<uintptr_t>(a.Y) & 31) == 0 && a.ldy % 16 == 0;
  const int64_t w_rows = static_cast<int64_t>(p.experts) * a.N * (kGated ? 2 : 1);
  // tiles, and rows of the tensor maps, are counted in 31 bits
  const int64_t tiles = (static_cast<int64_t>(a.M) / kRows + 1 + (kGrouped ? p.experts : 0)) * p.n_tiles;
  if (tiles >= (int64_t{1} << 31) || w_rows >= (int64_t{1} << 31)) return EPILORA_ERR_UNSUPPORTED;
  int rc = make_tma_2d_u8(&p.tmA, a.A, a.a_rows, a.K, a.K, kGrouped ? 1 : kRows, kBlock, true);
  if (rc == EPILORA_OK) rc = make_tma_2d_u8(&p.tmB, a.W, w_rows, a.K, a.K, kGated ? kRows : BN, kBlock, true);
  if (rc != EPILORA_OK) return rc;
  const int extra = 1024 + C::kMisc + (kGrouped ? 2 * (p.experts + 1) * 4 : 0);
  p.stages = (227 * 1024 - extra) / C::kStage;
  if (p.stages > C::kStagesMax) p.stages = C::kStagesMax;
  const int smem = p.stages * C::kStage + extra;
  const auto kern = block_gemm_kernel<BN, kGrouped, kGated>;
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

int launch_block_gemm(const BlockGemmArgs& a) {
  if (a.gated) return launch<256, true, true>(a);
  if (a.grouped) return launch<128, true, false>(a);
  return launch<128, false, false>(a);
}

}  // namespace epi
