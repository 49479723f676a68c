// Routing of tokens to experts: scores, an optional choice of groups, the
// best experts of a token and their weights. A warp per token, expert e in
// lane e % 32.
//
// The choice is by the exact order of score + bias, ties to the lowest index.
// The kernel works it out in 32 bits with a bound on what the roundings may
// have moved, and repeats a token in 64 bits where two candidates lie closer
// than that (FP64 is slow on this GPU; of random scores a few tokens in a
// thousand need it). Without a bias the order of the scores is the order of
// the logits, which needs no arithmetic.
//
// Bound: instructions and the chain of the choices; the bytes are few.
#include "blocks.cuh"
#include "ptx.cuh"

namespace epi {

namespace {

constexpr int kRouteThreads = 128;
constexpr unsigned kAll = 0xffffffffu;

template <class T>
__device__ __forceinline__ T neg_inf();
template <>
__device__ __forceinline__ float neg_inf<float>() { return __int_as_float(0xff800000); }
template <>
__device__ __forceinline__ double neg_inf<double>() { return __longlong_as_double(0xfff0000000000000ll); }

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

template <class T>
struct Best {
  T v;
  int i;
};
// largest value of the warp, the lowest index among equals
template <class T>
__device__ __forceinline__ Best<T> warp_best(Best<T> b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const T v = __shfl_xor_sync(kAll, b.v, o);
    const int i = __shfl_xor_sync(kAll, b.i, o);
    if (v > b.v || (v == b.v && i < b.i)) b = Best<T>{v, i};
  }
  return b;
}
template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// A logit as the scores take it: NaN counts as -infinity (no such expert),
// +infinity as the largest number.
__device__ __forceinline__ float clean(float l) {
  if (!(l > __int_as_float(0xff800000))) return __int_as_float(0xff800000);
  return fminf(l, 3.402823466e38f);
}

template <class T>
__device__ __forceinline__ T score_of(const MoeRouteArgs& a, float l, T top, T sum) {
  if (!(l > neg_inf<float>())) return T(0);
  if (a.sigmoid) return T(1) / (T(1) + exp_of(-T(l)));
  return exp_of(T(l) - top) / sum;
}

// Chooses the token's experts: slot j's in lane j (-1: none left). Returns
// whether two candidates were too close to tell (never for T = double).
template <class T, int kPer>
__device__ __forceinline__ bool choose(const MoeRouteArgs& a, const float (&l)[kPer], float top, int lane, int& mine) {
  constexpr bool kApprox = sizeof(T) == 4;
  const bool by_value = a.bias != nullptr || (a.groups > 1 && a.group_best > 1);
  T c[kPer], sum = T(1), bound = T(0);
  if (by_value && !a.sigmoid) {
    sum = T(0);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (l[i] > neg_inf<float>()) sum += exp_of(T(l[i]) - T(top));
    sum = warp_sum(sum);
  }
  T most = T(0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    c[i] = neg_inf<T>();
    if (e < a.experts && l[i] > neg_inf<float>()) {
      c[i] = by_value ? score_of<T>(a, l[i], T(top), sum) : T(l[i]);
      if (a.bias != nullptr) {
        c[i] += T(a.bias[e]);
        if (!(c[i] > neg_inf<T>())) c[i] = neg_inf<T>();      // (a NaN: no such expert)
      }
      if (kApprox && c[i] > neg_inf<T>() && c[i] < T(3e38)) most = c[i] < T(0) ? (most > -c[i] ? most : -c[i]) : (most > c[i] ? most : c[i]);
    }
  }
  if (kApprox && by_value) {
    // A sigmoid is off by a few units of 2^-24; a softmax by those of its
    // sum, at most 40 of them (additions in each lane, then five), and of
    // the exponent's argument (x e^x < 0.37). With the rounding of c itself,
    // 2^-24 of it; the difference of two, and of two sums of two.
    bound = (a.sigmoid ? T(0x1p-20) : T(0x1p-16)) + T(0x1p-21) * Best<T>(warp_best(Best<T>{most, 0})).v;
  }
  bool close = false;
  if (a.groups > 1 && a.top_groups < a.groups) {
    // lane g: the value of group g
    const int size = a.experts / a.groups;
    T value = neg_inf<T>();
    for (int g = 0; g < a.groups; ++g) {
      Best<T> first{neg_inf<T>(), 0x7fffffff};
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        if (e / size == g && c[i] > first.v) first = Best<T>{c[i], e};
      }
      first = warp_best(first);
      T v = first.v;
      if (a.group_best > 1 && v > neg_inf<T>()) {
        Best<T> second{neg_inf<T>(), 0x7fffffff};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = lane + 32 * i;
          if (e / size == g && e != first.i && c[i] > second.v) second = Best<T>{c[i], e};
        }
        second = warp_best(second);
        if (second.v > neg_inf<T>()) v += second.v;
      }
      if (lane == g) value = v;
    }
    unsigned kept = 0;
    T before = T(0);
    for (int j = 0; j <= a.top_groups; ++j) {
      const Best<T> b = warp_best(Best<T>{(kept >> lane) & 1u ? neg_inf<T>() : value, (kept >> lane) & 1u || lane >= a.groups ? 64 + lane : lane});
      if (kApprox && by_value && j == a.top_groups && b.v > neg_inf<T>() && !(before - b.v > bound)) close = true;
      before = b.v;
      if (j < a.top_groups && b.i < 32) kept |= 1u << b.i;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e < a.experts && !((kept >> (e / size)) & 1u)) c[i] = neg_inf<T>();
    }
  }
  // without a bias the experts themselves are told by their logits
  const bool by_logit = a.bias == nullptr;
  if (by_logit && by_value) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (c[i] > neg_inf<T>()) c[i] = T(l[i]);
  }
  mine = -1;
  T before = T(0);
  for (int j = 0; j <= a.top; ++j) {
    Best<T> b{neg_inf<T>(), 0x7fffffff};
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (c[i] > b.v) b = Best<T>{c[i], lane + 32 * i};
    b = warp_best(b);
    if (!(b.v > neg_inf<T>())) break;
    if (kApprox && !by_logit && j > 0 && !(before - b.v > bound)) close = true;
    before = b.v;
    if (j == a.top) break;
    if (lane == j) mine = b.i;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == b.i) c[i] = neg_inf<T>();
  }
  return close;
}

template <int kPer, bool kBf16>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const __grid_constant__ MoeRouteArgs a) {
  pdl_wait_primary();
  pdl_allow_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  float l[kPer], top = neg_inf<float>();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    l[i] = neg_inf<float>();
    if (e < a.experts)
      l[i] = clean(kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + e])
                         : static_cast<const float*>(a.logits)[t * a.ld + e]);
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  int mine;
  if (choose<float, kPer>(a, l, top, lane, mine)) choose<double, kPer>(a, l, top, lane, mine);
  // weights: the scores of the chosen, in 32 bits
  float sum = 1.0f;
  if (!a.sigmoid && !a.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (l[i] > neg_inf<float>()) sum += expf(l[i] - top);
    sum = warp_sum(sum);
  }
  float lm = neg_inf<float>();
  if (mine >= 0)
    lm = clean(kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + mine])
                     : static_cast<const float*>(a.logits)[t * a.ld + mine]);
  if (a.renormalize) {
    // softmax: against the largest of the chosen, whose scores may all be too
    // small for 32 bits; a sigmoid of less than -30 is e^x within 2^-43 of it
    top = lm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  }
  float w = 0.0f;
  if (mine >= 0)
    w = a.sigmoid && !(a.renormalize && top < -30.0f) ? 1.0f / (1.0f + expf(-lm)) : expf(lm - top) / sum;
  if (a.renormalize) {
    const float all = warp_sum(w);
    w = all > 0.0f ? w / all : 0.0f;
  }
  if (lane < a.top) {
    a.ids[t * a.top + lane] = mine;
    a.weights[t * a.top + lane] = w * a.scale;
  }
}

template <int kPer>
int launch(const MoeRouteArgs& a) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.tokens) + kRouteThreads / 32 - 1) / (kRouteThreads / 32));
  return a.bf16 ? launch_dependent(moe_route_kernel<kPer, true>, grid, kRouteThreads, 0, a.stream, a)
                : launch_dependent(moe_route_kernel<kPer, false>, grid, kRouteThreads, 0, a.stream, a);
}

}  // namespace

int launch_moe_route(const MoeRouteArgs& a) {
  if (a.experts <= 64) return launch<2>(a);
  if (a.experts <= 128) return launch<4>(a);
  if (a.experts <= 256) return launch<8>(a);
  if (a.experts <= 512) return launch<16>(a);
  return launch<32>(a);
}

}  // namespace epi
