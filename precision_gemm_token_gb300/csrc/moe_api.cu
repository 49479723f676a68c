// C ABI of the operators in 8-bit blocks and of the mixture-of-experts
// operators: argument validation and workspace layout.
#include <atomic>
#include <cmath>

#include "blocks.cuh"

using namespace epi;

namespace {

std::atomic<int> g_late_copies{0};

inline bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool there(const void* p, size_t n) { return p != nullptr && al(p, n); }
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }
inline bool width_ok(int k) { return k >= 16 && k % 16 == 0; }

// beyond this, sums of a size and a tile's would not fit 32 bits
inline bool too_large(int a, int b, int c = 0) {
  return a > EPILORA_BLOCK_MAX_SIZE || b > EPILORA_BLOCK_MAX_SIZE || c > EPILORA_BLOCK_MAX_SIZE;
}

bool quant_ok(const void* X, int M, int K, int64_t ldx) {
  return M >= 0 && width_ok(K) && ldx >= K && ldx % 8 == 0 && (M == 0 || there(X, 16));
}

// what the calls cut off their workspace
struct Cut {
  uint8_t* at;
  size_t used = 0;
  explicit Cut(void* ws) : at(static_cast<uint8_t*>(ws)) {}
  template <class T>
  T* take(size_t n) {
    T* p = reinterpret_cast<T*>(at + used);
    used += round256(n * sizeof(T));
    return p;
  }
};

struct Parts {
  MoePlan plan;
  uint8_t *xq, *inner;           // by row
  float *x_scale, *inner_scale;
  void* out;                     // by slot, fp32 with EPILORA_MOE_F32_PARTS, else bf16
  size_t bytes;
};
Parts cut_moe(void* ws, int what, int tokens, int top, int experts, int hidden, int inner) {
  Cut c(ws);
  Parts p{};
  const size_t slots = static_cast<size_t>(tokens) * top;
  p.plan.offsets = c.take<int32_t>(experts + 1);
  p.plan.slots = c.take<int32_t>(slots);
  p.plan.rows = c.take<int32_t>(slots);
  if (what & EPILORA_MOE_UP) {
    p.xq = c.take<uint8_t>(slots * hidden);
    p.x_scale = c.take<float>(n_blocks(hidden) * slots);
  }
  if (what & EPILORA_MOE_DOWN) {
    p.inner = c.take<uint8_t>(slots * inner);
    p.inner_scale = c.take<float>(n_blocks(inner) * slots);
    p.out = c.take<uint8_t>(slots * hidden * (what & EPILORA_MOE_F32_PARTS ? sizeof(float) : sizeof(uint16_t)));
  }
  p.bytes = c.used;
  return p;
}

// sizes of a mixture: EPILORA_OK, or the refusal
int moe_sizes(int tokens, int top, int experts, int hidden, int inner) {
  if (tokens < 0 || top < 1 || experts < 1 || !width_ok(hidden) || !width_ok(inner)) return EPILORA_ERR_INVALID_ARG;
  if (experts > EPILORA_MOE_MAX_EXPERTS || too_large(hidden, inner) || static_cast<int64_t>(tokens) * top >= (int64_t{1} << 30))
    return EPILORA_ERR_UNSUPPORTED;
  return EPILORA_OK;
}

struct MoeCall {
  int tokens, top, experts, hidden, inner;
  const int32_t* ids;
  int* status;
  cudaStream_t stream;
};

int enqueue_plan(const MoeCall& m, const Parts& p) {
  return launch_moe_plan(MoePlanArgs{m.ids, m.tokens, m.top, m.experts, p.plan, m.status, m.stream});
}

// (by_slot: the output in the order of the slots, zeros where there is no expert)
int enqueue_up(const MoeCall& m, const Parts& p, const void* X, int64_t ldx, const uint8_t* W, const float* w_scale,
               uint8_t* inner, float* inner_scale, bool by_slot) {
  const int slots = m.tokens * m.top;
  MoeScatterArgs s{};
  s.q = BlockQuantArgs{X, m.tokens, m.hidden, ldx, p.xq, p.x_scale, slots, m.stream};
  s.top = m.top;
  s.rows = p.plan.rows;
  s.inner = by_slot ? inner : nullptr;
  s.inner_scale = inner_scale;
  s.inner_dim = m.inner;
  const int rc = launch_moe_scatter(s);
  if (rc != EPILORA_OK) return rc;
  BlockGemmArgs g{};
  g.M = slots;
  g.N = m.inner;
  g.K = m.hidden;
  g.A = p.xq;
  g.a_scale = p.x_scale;
  g.a_scale_ld = slots;
  g.W = W;
  g.w_scale = w_scale;
  g.grouped = g.gated = 1;
  g.experts = m.experts;
  g.offsets = p.plan.offsets;
  g.out_rows = by_slot ? p.plan.slots : nullptr;
  g.inner = inner;
  g.inner_scale = inner_scale;
  g.status = m.status;
  g.stream = m.stream;
  return launch_block_gemm(g);
}

// from p.inner, by row
int enqueue_down(const MoeCall& m, const Parts& p, int f32, const uint8_t* W, const float* w_scale,
                 const float* weights, void* Y, int64_t ldy) {
  BlockGemmArgs g{};
  g.M = m.tokens * m.top;
  g.N = m.hidden;
  g.K = m.inner;
  g.A = p.inner;
  g.a_scale = p.inner_scale;
  g.a_scale_ld = g.M;
  g.W = W;
  g.w_scale = w_scale;
  g.Y = p.out;
  g.f32 = f32;
  g.ldy = m.hidden;
  g.grouped = 1;
  g.experts = m.experts;
  g.offsets = p.plan.offsets;
  g.out_rows = p.plan.slots;
  g.status = m.status;
  g.stream = m.stream;
  const int rc = launch_block_gemm(g);
  if (rc != EPILORA_OK) return rc;
  return launch_moe_combine(
      MoeCombineArgs{m.ids, weights, m.tokens, m.top, m.experts, m.hidden, p.out, f32, Y, ldy, m.stream});
}

bool out_ok(const void* Y, int64_t ldy, int hidden) { return there(Y, 16) && ldy >= hidden && ldy % 8 == 0; }
bool ws_ok(const void* ws, size_t bytes, size_t need) { return there(ws, 256) && bytes >= need; }

size_t moe_bytes(int what, int tokens, int top, int experts, int hidden, int inner) {
  return cut_moe(nullptr, what, tokens, top, experts, hidden, inner).bytes;
}

// f32: the experts' outputs stay fp32 until their sum
int experts_down(int tokens, int top, int experts, int hidden, int inner, const uint8_t* Hq, const float* h_scale,
                 const int32_t* ids, const float* weights, const uint8_t* Wdown, const float* wdown_scale, void* Y,
                 int64_t ldy, void* workspace, size_t workspace_bytes, int* status_dev, void* stream, int f32) {
  const int what = EPILORA_MOE_DOWN | (f32 ? EPILORA_MOE_F32_PARTS : 0);
  int rc = moe_sizes(tokens, top, experts, hidden, inner);
  if (rc != EPILORA_OK) return rc;
  if (tokens == 0) return EPILORA_OK;
  if (!there(Hq, 16) || !there(h_scale, 4) || !there(ids, 4) || !there(weights, 4) || !there(Wdown, 16) ||
      !there(wdown_scale, 4) || !out_ok(Y, ldy, hidden) || !al(status_dev, 4))
    return EPILORA_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, moe_bytes(what, tokens, top, experts, hidden, inner)))
    return EPILORA_ERR_WORKSPACE;
  const Parts p = cut_moe(workspace, what, tokens, top, experts, hidden, inner);
  const MoeCall m{tokens, top, experts, hidden, inner, ids, status_dev, static_cast<cudaStream_t>(stream)};
  rc = enqueue_plan(m, p);
  if (rc == EPILORA_OK)
    rc = launch_moe_gather(
        MoeGatherArgs{Hq, h_scale, p.inner, p.inner_scale, tokens * top, inner, p.plan.rows, m.stream});
  return rc != EPILORA_OK ? rc : enqueue_down(m, p, f32, Wdown, wdown_scale, weights, Y, ldy);
}

int experts_both(int tokens, int top, int experts, int hidden, int inner, const void* X, int64_t ldx,
                 const int32_t* ids, const float* weights, const uint8_t* Wup, const float* wup_scale,
                 const uint8_t* Wdown, const float* wdown_scale, void* Y, int64_t ldy, void* workspace,
                 size_t workspace_bytes, int* status_dev, void* stream, int f32) {
  const int what = EPILORA_MOE_UP | EPILORA_MOE_DOWN | (f32 ? EPILORA_MOE_F32_PARTS : 0);
  int rc = moe_sizes(tokens, top, experts, hidden, inner);
  if (rc != EPILORA_OK) return rc;
  if (!quant_ok(X, tokens, hidden, ldx)) return EPILORA_ERR_INVALID_ARG;
  if (tokens == 0) return EPILORA_OK;
  if (!there(ids, 4) || !there(weights, 4) || !there(Wup, 16) || !there(wup_scale, 4) || !there(Wdown, 16) ||
      !there(wdown_scale, 4) || !out_ok(Y, ldy, hidden) || !al(status_dev, 4))
    return EPILORA_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, moe_bytes(what, tokens, top, experts, hidden, inner)))
    return EPILORA_ERR_WORKSPACE;
  const Parts p = cut_moe(workspace, what, tokens, top, experts, hidden, inner);
  const MoeCall m{tokens, top, experts, hidden, inner, ids, status_dev, static_cast<cudaStream_t>(stream)};
  rc = enqueue_plan(m, p);
  if (rc == EPILORA_OK) rc = enqueue_up(m, p, X, ldx, Wup, wup_scale, p.inner, p.inner_scale, false);
  return rc != EPILORA_OK ? rc : enqueue_down(m, p, f32, Wdown, wdown_scale, weights, Y, ldy);
}

}  // namespace

int epi::block_test_late_copies() { return g_late_copies.load(); }

extern "C" {

EPILORA_API int epilora_block_quant(const void* X, int M, int K, int64_t ldx, uint8_t* Xq, float* x_scale,
                                    int64_t x_scale_ld, void* stream) {
  if (!quant_ok(X, M, K, ldx) || x_scale_ld < M) return EPILORA_ERR_INVALID_ARG;
  if (too_large(M, K)) return EPILORA_ERR_UNSUPPORTED;
  if (M == 0) return EPILORA_OK;
  if (!there(Xq, 16) || !there(x_scale, 4)) return EPILORA_ERR_INVALID_ARG;
  return launch_block_quant(
      BlockQuantArgs{X, M, K, ldx, Xq, x_scale, x_scale_ld, static_cast<cudaStream_t>(stream)});
}

EPILORA_API int epilora_block_quant_weight(const void* W, int N, int K, int64_t ldw, uint8_t* Wq, float* w_scale,
                                           void* stream) {
  if (!quant_ok(W, N, K, ldw)) return EPILORA_ERR_INVALID_ARG;
  if (too_large(N, K)) return EPILORA_ERR_UNSUPPORTED;
  if (N == 0) return EPILORA_OK;
  if (!there(Wq, 16) || !there(w_scale, 4)) return EPILORA_ERR_INVALID_ARG;
  return launch_block_quant_weight(W, N, K, ldw, Wq, w_scale, static_cast<cudaStream_t>(stream));
}

EPILORA_API int epilora_block_matmul(int M, int N, int K, const uint8_t* Xq, const float* x_scale, int64_t x_scale_ld,
                                     const uint8_t* Wq, const float* w_scale, void* Y, int64_t ldy, int* status_dev,
                                     void* stream) {
  if (M < 0 || N < 1 || !width_ok(K) || x_scale_ld < M || ldy < N) return EPILORA_ERR_INVALID_ARG;
  if (too_large(M, N, K)) return EPILORA_ERR_UNSUPPORTED;
  if (M == 0) return EPILORA_OK;
  if (!there(Xq, 16) || !there(x_scale, 4) || !there(Wq, 16) || !there(w_scale, 4) || !there(Y, 2) || !al(status_dev, 4))
    return EPILORA_ERR_INVALID_ARG;
  BlockGemmArgs g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.A = Xq;
  g.a_scale = x_scale;
  g.a_scale_ld = x_scale_ld;
  g.W = Wq;
  g.w_scale = w_scale;
  g.Y = Y;
  g.ldy = ldy;
  g.status = status_dev;
  g.stream = static_cast<cudaStream_t>(stream);
  return launch_block_gemm(g);
}

EPILORA_API int epilora_test_late_block_copies(int on) {
  g_late_copies.store(on != 0 ? 1 : 0);
  return EPILORA_OK;
}

EPILORA_API size_t epilora_block_linear_workspace_bytes(int M, int K) {
  if (M < 0 || !width_ok(K) || too_large(M, K)) return 0;
  return round256(static_cast<size_t>(M) * K) + round256(static_cast<size_t>(n_blocks(K)) * M * sizeof(float));
}

EPILORA_API int epilora_block_linear(int M, int N, int K, const void* X, int64_t ldx, const uint8_t* Wq,
                                     const float* w_scale, void* Y, int64_t ldy, void* workspace,
                                     size_t workspace_bytes, int* status_dev, void* stream) {
  if (N < 1 || ldy < N || !quant_ok(X, M, K, ldx)) return EPILORA_ERR_INVALID_ARG;
  if (too_large(M, N, K)) return EPILORA_ERR_UNSUPPORTED;
  if (M == 0) return EPILORA_OK;
  if (!there(Wq, 16) || !there(w_scale, 4) || !there(Y, 2) || !al(status_dev, 4)) return EPILORA_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, epilora_block_linear_workspace_bytes(M, K))) return EPILORA_ERR_WORKSPACE;
  Cut c(workspace);
  uint8_t* xq = c.take<uint8_t>(static_cast<size_t>(M) * K);
  float* xs = c.take<float>(static_cast<size_t>(n_blocks(K)) * M);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rc = launch_block_quant(BlockQuantArgs{X, M, K, ldx, xq, xs, M, s});
  if (rc != EPILORA_OK) return rc;
  BlockGemmArgs g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.A = xq;
  g.a_scale = xs;
  g.a_scale_ld = M;
  g.W = Wq;
  g.w_scale = w_scale;
  g.Y = Y;
  g.ldy = ldy;
  g.early_weights = 1;      // (the quantizer lets this kernel start only once everything before it is done)
  g.status = status_dev;
  g.stream = s;
  return launch_block_gemm(g);
}

EPILORA_API int epilora_moe_route(int tokens, int experts, int top, const void* logits, int logits_fmt, int64_t ld,
                                  const float* bias, int scoring, int groups, int top_groups, int group_best,
                                  int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
  if (tokens < 0 || experts < 1 || top < 1 || ld < experts || !std::isfinite(scale)) return EPILORA_ERR_INVALID_ARG;
  if (logits_fmt != EPILORA_LOGITS_F32 && logits_fmt != EPILORA_LOGITS_BF16) return EPILORA_ERR_INVALID_ARG;
  if (scoring != EPILORA_SCORE_SOFTMAX && scoring != EPILORA_SCORE_SIGMOID) return EPILORA_ERR_INVALID_ARG;
  if (groups < 1 || experts % groups != 0 || top_groups < 1 || top_groups > groups || group_best < 1 || group_best > 2)
    return EPILORA_ERR_INVALID_ARG;
  if (top > experts / groups * top_groups) return EPILORA_ERR_INVALID_ARG;
  if (experts > EPILORA_MOE_MAX_EXPERTS || top > EPILORA_MOE_MAX_TOP || groups > 32) return EPILORA_ERR_UNSUPPORTED;
  if (tokens == 0) return EPILORA_OK;
  if (!there(logits, logits_fmt == EPILORA_LOGITS_F32 ? 4 : 2) || !al(bias, 4) || !there(ids, 4) || !there(weights, 4))
    return EPILORA_ERR_INVALID_ARG;
  MoeRouteArgs a{};
  a.logits = logits;
  a.bf16 = logits_fmt == EPILORA_LOGITS_BF16;
  a.tokens = tokens;
  a.experts = experts;
  a.top = top;
  a.ld = ld;
  a.bias = bias;
  a.sigmoid = scoring == EPILORA_SCORE_SIGMOID;
  a.groups = groups;
  a.top_groups = top_groups;
  a.group_best = group_best;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_moe_route(a);
}

EPILORA_API size_t epilora_moe_workspace_bytes(int what, int tokens, int top, int experts, int hidden, int inner) {
  constexpr int kAll = EPILORA_MOE_UP | EPILORA_MOE_DOWN | EPILORA_MOE_F32_PARTS;
  // (the parts are those of down)
  if (what < EPILORA_MOE_UP || what > kAll || ((what & EPILORA_MOE_F32_PARTS) && !(what & EPILORA_MOE_DOWN)) ||
      moe_sizes(tokens, top, experts, hidden, inner) != EPILORA_OK)
    return 0;
  return moe_bytes(what, tokens, top, experts, hidden, inner);
}

EPILORA_API int epilora_moe_experts_up(int tokens, int top, int experts, int hidden, int inner, const void* X,
                                       int64_t ldx, const int32_t* ids, const uint8_t* Wup, const float* wup_scale,
                                       uint8_t* Hq, float* h_scale, void* workspace, size_t workspace_bytes,
                                       int* status_dev, void* stream) {
  int rc = moe_sizes(tokens, top, experts, hidden, inner);
  if (rc != EPILORA_OK) return rc;
  if (!quant_ok(X, tokens, hidden, ldx)) return EPILORA_ERR_INVALID_ARG;
  if (tokens == 0) return EPILORA_OK;
  if (!there(ids, 4) || !there(Wup, 16) || !there(wup_scale, 4) || !there(Hq, 16) || !there(h_scale, 4) ||
      !al(status_dev, 4))
    return EPILORA_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, moe_bytes(EPILORA_MOE_UP, tokens, top, experts, hidden, inner)))
    return EPILORA_ERR_WORKSPACE;
  const Parts p = cut_moe(workspace, EPILORA_MOE_UP, tokens, top, experts, hidden, inner);
  const MoeCall m{tokens, top, experts, hidden, inner, ids, status_dev, static_cast<cudaStream_t>(stream)};
  rc = enqueue_plan(m, p);
  return rc != EPILORA_OK ? rc : enqueue_up(m, p, X, ldx, Wup, wup_scale, Hq, h_scale, true);
}

EPILORA_API int epilora_moe_experts_down(int tokens, int top, int experts, int hidden, int inner, const uint8_t* Hq,
                                         const float* h_scale, const int32_t* ids, const float* weights,
                                         const uint8_t* Wdown, const float* wdown_scale, void* Y, int64_t ldy,
                                         void* workspace, size_t workspace_bytes, int* status_dev, void* stream) {
  return experts_down(tokens, top, experts, hidden, inner, Hq, h_scale, ids, weights, Wdown, wdown_scale, Y, ldy,
                      workspace, workspace_bytes, status_dev, stream, 0);
}

EPILORA_API int epilora_moe_experts_down_f32(int tokens, int top, int experts, int hidden, int inner, const uint8_t* Hq,
                                             const float* h_scale, const int32_t* ids, const float* weights,
                                             const uint8_t* Wdown, const float* wdown_scale, void* Y, int64_t ldy,
                                             void* workspace, size_t workspace_bytes, int* status_dev, void* stream) {
  return experts_down(tokens, top, experts, hidden, inner, Hq, h_scale, ids, weights, Wdown, wdown_scale, Y, ldy,
                      workspace, workspace_bytes, status_dev, stream, 1);
}

EPILORA_API int epilora_moe_experts(int tokens, int top, int experts, int hidden, int inner, const void* X, int64_t ldx,
                                    const int32_t* ids, const float* weights, const uint8_t* Wup,
                                    const float* wup_scale, const uint8_t* Wdown, const float* wdown_scale, void* Y,
                                    int64_t ldy, void* workspace, size_t workspace_bytes, int* status_dev,
                                    void* stream) {
  return experts_both(tokens, top, experts, hidden, inner, X, ldx, ids, weights, Wup, wup_scale, Wdown, wdown_scale, Y,
                      ldy, workspace, workspace_bytes, status_dev, stream, 0);
}

EPILORA_API int epilora_moe_experts_f32(int tokens, int top, int experts, int hidden, int inner, const void* X,
                                        int64_t ldx, const int32_t* ids, const float* weights, const uint8_t* Wup,
                                        const float* wup_scale, const uint8_t* Wdown, const float* wdown_scale, void* Y,
                                        int64_t ldy, void* workspace, size_t workspace_bytes, int* status_dev,
                                        void* stream) {
  return experts_both(tokens, top, experts, hidden, inner, X, ldx, ids, weights, Wup, wup_scale, Wdown, wdown_scale, Y,
                      ldy, workspace, workspace_bytes, status_dev, stream, 1);
}

}  // extern "C"
