// Routing of tokens to experts: scores, an optional choice of groups, the
// best experts of a token and their weights. A warp per token, expert e in
// lane e % 32.
//
// The choice is by score + bias in 64 bits; where those are equal (a sigmoid
// that is 1 there, a softmax's score below the last bit of its bias) the larger
// logit goes first, which with equal biases is the order of the real numbers,
// then the lowest index. The kernel works it out in 32 bits with a bound on
// what the roundings may have moved. Where two candidates lie closer than that
// (of random scores, in 1 to 20 of 1000 tokens: more, the more experts and the
// more of them chosen) it looks at them in 64 bits: of a sigmoid's chosen
// experts a lane each, else the whole token again (FP64 is slow on this GPU:
// 20 us for such a token, which then is the call's time). Without a bias the
// order of the scores is the order of the logits, which needs no arithmetic.
//
// Bound: the chain of the choices (4096 x 256 with eight groups: some 30 maxima over the warp a token, 18.4 us; one
// token of 128 experts 3 us); the bytes are few. Softmax with a bias: of 4096
// tokens some go through 64 bits again, 27 us of 256 experts, 65 of 512 with 16
// chosen (without a bias 18).
#include "blocks.cuh"
#include "ptx.cuh"

namespace epi {

namespace {

constexpr int kRouteThreads = 128;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }

// Numbers as unsigned keys of the same order (the order of the bits, turned
// round for negative numbers): maxima over the warp by redux, and 64-bit
// comparisons without the FP64 pipe. Key 0: nobody (no number has it).
template <class T>
struct Keys;
template <>
struct Keys<float> {
  typedef uint32_t Key;
  static __device__ __forceinline__ Key of(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
  }
  static __device__ __forceinline__ float value(Key k) {
    return __uint_as_float((k & 0x80000000u) != 0 ? k & 0x7fffffffu : ~k);
  }
  static __device__ __forceinline__ Key warp_max(Key k) { return __reduce_max_sync(kAll, k); }
};
template <>
struct Keys<double> {
  typedef uint64_t Key;
  static __device__ __forceinline__ Key of(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    return (b >> 63) != 0 ? ~b : b | (1ull << 63);
  }
  static __device__ __forceinline__ double value(Key k) {
    return __longlong_as_double(static_cast<long long>((k >> 63) != 0 ? k & ~(1ull << 63) : ~k));
  }
  static __device__ __forceinline__ Key warp_max(Key k) {
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
  }
};

// The warp's largest key, and the lowest index that has it.
template <class T>
struct Best {
  typename Keys<T>::Key key;
  int i;
};
template <class T>
__device__ __forceinline__ Best<T> warp_best(Best<T> mine) {
  const typename Keys<T>::Key key = Keys<T>::warp_max(mine.key);
  return Best<T>{key, static_cast<int>(__reduce_min_sync(kAll, mine.key == key ? static_cast<uint32_t>(mine.i) : 0x7fffffffu))};
}
// The same where equal keys go by `logit` (that of `mine`) first.
template <class T>
__device__ __forceinline__ Best<T> warp_best(Best<T> mine, float logit) {
  const typename Keys<T>::Key key = Keys<T>::warp_max(mine.key);
  const uint32_t l = mine.key == key ? Keys<float>::of(logit) : 0u;
  const uint32_t most = __reduce_max_sync(kAll, l);        // (by all lanes, whatever their keys)
  const bool best = mine.key == key && l == most;
  return Best<T>{key, static_cast<int>(__reduce_min_sync(kAll, best ? static_cast<uint32_t>(mine.i) : 0x7fffffffu))};
}
__device__ __forceinline__ float warp_max(float v) {      // of numbers that are not negative
  return __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(v)));
}
template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// A logit as the scores take it: NaN counts as -infinity (no such expert),
// +infinity as the largest number, -0 as 0.
__device__ __forceinline__ float clean(float l) {
  if (!(l > minus_inf())) return minus_inf();
  return fminf(l, 3.402823466e38f) + 0.0f;
}

// Chooses the token's experts: slot j's in lane j (-1: none left). Returns
// what is too close to tell (nothing for T = double): kGroups, of the groups
// or of more experts than there are lanes; kExperts, of the chosen experts,
// and then the lanes have all candidates for them, `top` or more.
enum : int { kTold = 0, kExperts = 1, kGroups = 2 };
template <class T, int kPer>
__device__ __forceinline__ int choose(const MoeRouteArgs& a, const float (&l)[kPer], float top, int lane, int& mine) {
  typedef typename Keys<T>::Key Key;
  constexpr bool kApprox = sizeof(T) == 4;
  const bool by_value = a.bias != nullptr || (a.groups > 1 && a.group_best > 1);
  Key c[kPer];
  T sum = T(1);
  // what roundings may do to the difference of two scores, or of two sums of two (below)
  if (by_value && !a.sigmoid) {
    sum = T(0);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (l[i] > minus_inf()) sum += exp_of(T(l[i]) - T(top));
    sum = warp_sum(sum);
  }
  float most = 0.0f, largest = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    c[i] = 0;
    if (e < a.experts && l[i] > minus_inf()) {
      T v = T(l[i]);
      if (by_value) v = a.sigmoid ? T(1) / (T(1) + exp_of(-v)) : exp_of(v - T(top)) / sum;
      if (kApprox) largest = fmaxf(largest, static_cast<float>(v));
      if (a.bias != nullptr) v += T(a.bias[e]);
      if (v > T(minus_inf())) c[i] = Keys<T>::of(v);      // (a bias of -infinity or NaN: no such expert)
      if (kApprox && fabsf(static_cast<float>(v)) < 3e38f) most = fmaxf(most, fabsf(static_cast<float>(v)));
    }
  }
  // In units u = 2^-24: a sigmoid is off by 2.5. A softmax's score is off, in u
  // of the largest (1 / sum), by 4.4 for the exponential (two of its own steps,
  // and the rounded argument, |x| e^x < 0.37), 36 for the additions of the sum
  // (31 in a lane, then five), 11 for its terms (their mean |x| is at most
  // ln 1024) and 1 for the quotient: 53. The rounding of c itself is 1 of it;
  // the difference of two sums of two has four times all that.
  T bound = T(0);
  if (kApprox && by_value)
    bound = T((a.sigmoid ? 0x1p-20f : 0x1p-16f * warp_max(largest)) + 0x1p-21f * warp_max(most));
  int close = kTold;
  if (a.groups > 1 && a.top_groups < a.groups) {
    const int size = a.experts / a.groups;
    int group[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) group[i] = (lane + 32 * i) / size;
    Key value = 0;                                        // lane g: of group g
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      Best<T> first{0, 0x7fffffff};
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (group[i] == g && c[i] > first.key) first = Best<T>{c[i], lane + 32 * i};
      first = warp_best(first);
      Key v = first.key;
      if (a.group_best > 1 && v != 0) {
        Key second = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (group[i] == g && lane + 32 * i != first.i && c[i] > second) second = c[i];
        second = Keys<T>::warp_max(second);
        if (second != 0) v = Keys<T>::of(Keys<T>::value(v) + Keys<T>::value(second));
      }
      if (lane == g) value = v;
    }
    unsigned kept = 0;
    Key before = 0;
#pragma unroll 1
    for (int j = 0; j <= a.top_groups; ++j) {
      // (a group that nobody is in is still there to be kept, after the others)
      const bool there = lane < a.groups && ((kept >> lane) & 1u) == 0;
      const Best<T> b = warp_best(Best<T>{there ? value : 0, there ? lane : 0x7fffffff});
      if (kApprox && by_value && j == a.top_groups && b.key != 0 &&
          !(Keys<T>::value(before) - Keys<T>::value(b.key) > bound))
        close = kGroups;
      before = b.key;
      if (j < a.top_groups) kept |= 1u << b.i;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (((kept >> (group[i] & 31)) & 1u) == 0) c[i] = 0;
  }
  // without a bias the experts themselves are told by their logits
  const bool by_logit = a.bias == nullptr;
  if (by_logit && by_value) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (c[i] != 0) c[i] = Keys<T>::of(T(l[i]));
  }
  mine = -1;
  Key before = 0;
#pragma unroll 1
  for (int j = 0;; ++j) {
    Best<T> b{0, 0x7fffffff};
    if constexpr (kApprox) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c[i] > b.key) b = Best<T>{c[i], lane + 32 * i};
      b = warp_best(b);
    } else {
      float logit = minus_inf();
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c[i] > b.key || (c[i] == b.key && c[i] != 0 && l[i] > logit)) {
          b = Best<T>{c[i], lane + 32 * i};
          logit = l[i];
        }
      b = warp_best(b, logit);
    }
    if (b.key == 0) break;
    const bool near = kApprox && !by_logit && j > 0 && !(Keys<T>::value(before) - Keys<T>::value(b.key) > bound);
    if (j >= a.top && !near) break;
    if (near) close = max(close, static_cast<int>(kExperts));
    if (j == 32) {
      close = kGroups;
      break;
    }
    before = b.key;
    if (lane == j) mine = b.i;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == b.i) c[i] = 0;
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
  const auto logit = [&](int e) {
    return clean(kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + e])
                       : static_cast<const float*>(a.logits)[t * a.ld + e]);
  };
  float l[kPer], top = minus_inf();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    l[i] = minus_inf();
    if (e < a.experts)
      l[i] = logit(e);
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  int mine;
  const int close = choose<float, kPer>(a, l, top, lane, mine);
  if (close == kExperts && a.sigmoid) {
    // the candidates in 64 bits, a lane each, and their order
    const float at = mine < 0 ? minus_inf() : logit(mine);
    const Keys<double>::Key key =
        mine < 0 ? 0 : Keys<double>::of(1.0 / (1.0 + exp(-static_cast<double>(at))) + static_cast<double>(a.bias[mine]));
    int before = 0, told = -1;
    for (int o = 0; o < 32; ++o) {
      const Keys<double>::Key k = __shfl_sync(kAll, key, o);
      const float le = __shfl_sync(kAll, at, o);
      const int e = __shfl_sync(kAll, mine, o);
      if (k > key || (k == key && (le > at || (le == at && e < mine)))) ++before;
    }
    for (int j = 0; j < a.top; ++j) {
      const unsigned who = __ballot_sync(kAll, mine >= 0 && before == j);
      const int e = __shfl_sync(kAll, mine, who != 0 ? __ffs(who) - 1 : 0);
      if (lane == j && who != 0) told = e;
    }
    mine = told;
  } else if (close != kTold) {
    choose<double, kPer>(a, l, top, lane, mine);
  }
  // weights: the scores of the chosen, in 32 bits
  float sum = 1.0f;
  if (!a.sigmoid && !a.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (l[i] > minus_inf()) sum += expf(l[i] - top);
    sum = warp_sum(sum);
  }
  float lm = minus_inf();
  if (mine >= 0) lm = logit(mine);
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
