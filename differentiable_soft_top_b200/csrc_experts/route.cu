// route.cu -- the choice of experts and its gradient.
//
// One warp per token: lane l holds experts l, l + 32, ..; a choice is one
// integer maximum over the warp (keys mapped to integers of the same order)
// and one minimum over the indices that reach it.  The floor is the scores'
// bytes; what bounds it is the issue of the k rounds.
//
// Equal results whatever the rounding: without a bias and without sums of two
// keys the order of the keys is the order of the scores, which are compared as
// they are.  Otherwise fp32 keys decide only when neighbours in the order lie
// further apart than the fp32 error can reach; a token where they do not is
// done again with fp64 keys (about 1 in 1000 at 256 experts).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.h"

namespace lapsum {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;

template <int kDtype>
__device__ __forceinline__ float load_score(const void* p, int64_t i) {
  if (kDtype == LAPSUM_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t u = __ldg(static_cast<const uint16_t*>(p) + i);
  return kDtype == LAPSUM_BF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}
template <int kDtype>
__device__ __forceinline__ void store_score(void* p, int64_t i, float v) {
  if (kDtype == LAPSUM_F32)
    static_cast<float*>(p)[i] = v;
  else if (kDtype == LAPSUM_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <typename K>
__device__ __forceinline__ K warp_sum(K v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// integers in the order of the keys; 0 is below every key
__device__ __forceinline__ uint32_t ordered(float f) {
  uint32_t u = __float_as_uint(f);
  u = u == 0x80000000u ? 0u : u;  // -0 as +0 (an addition would flush subnormals)
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);  // -0 as +0
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float key_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ double key_of(uint64_t o) {
  return __longlong_as_double((int64_t)(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}
__device__ __forceinline__ uint32_t warp_top(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_top(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

struct Rule {
  int experts, k, score;
  int groups, size, kept, top;  // size: experts of a group
  bool raw;                     // the scores themselves are in the order of the keys
};

template <typename K>
struct Order {
  using O = uint32_t;
};
template <>
struct Order<double> {
  using O = uint64_t;
};

// What the order of a token's keys rests on; the fp32 bounds need the largest
// bias and, for scores used as they are, the largest score.
struct Keys {
  const void* scores;
  int64_t at;         // the token's first score
  const float* bias;
  float bias_max;
};

// Lane j < k gets the token's j-th choice (or -1).  l: this lane's scores, -inf
// where masked; b: its biases.  Returns whether the choice is certain at the
// precision of K (always, for fp64 and for raw keys).
template <typename K, int kDtype, int kPer>
__device__ __forceinline__ bool choose(const Rule& r, const Keys& in, const float (&l)[kPer], const float (&b)[kPer],
                                       int& mine) {
  using O = typename Order<K>::O;
  constexpr bool kCheck = sizeof(K) == 4;
  const int lane = threadIdx.x & 31;
  O o[kPer];
  bool certain = true;
  if (r.raw) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = l[i] == -INFINITY ? O(0) : ordered((K)l[i]);
  } else {
    K top = 0, total = 1;
    if (r.score == LAPSUM_SCORE_SOFTMAX) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = fmaxf(m, l[i]);
      top = (K)warp_max(m);
      K s = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (l[i] != -INFINITY) s += exp_of((K)l[i] - top);
      total = warp_sum(s);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      K s = (K)l[i];
      if (r.score == LAPSUM_SCORE_SOFTMAX) s = exp_of(s - top) / total;
      if (r.score == LAPSUM_SCORE_SIGMOID) s = (K)1 / ((K)1 + exp_of(-s));
      o[i] = l[i] == -INFINITY ? O(0) : ordered(s + (K)b[i]);
    }
  }
  if (r.groups > 1) {
    K value = -INFINITY;  // lane g: the value of group g
    for (int g = 0; g < r.groups; ++g) {
      const int e0 = g * r.size, e1 = e0 + r.size;
      O best = 0;
      int at = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = i * 32 + lane;
        if (e >= e0 && e < e1 && o[i] > best) {
          best = o[i];
          at = i;
        }
      }
      const O first = warp_top(best);
      K v = first ? key_of(first) : (K)-INFINITY;
      if (r.top == 2 && first) {
        const int who = __ffs(__ballot_sync(kAll, best == first)) - 1;
        O second = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = i * 32 + lane;
          if (e >= e0 && e < e1 && !(i == at && lane == who)) second = max(second, o[i]);
        }
        second = warp_top(second);
        if (second) v += key_of(second);
      }
      if (lane == g) value = v;
    }
    int above = 0;
    for (int g = 0; g < r.groups; ++g) {
      const K v = __shfl_sync(kAll, value, g);
      above += (v > value || (v == value && g < lane)) ? 1 : 0;
    }
    const uint32_t stay = __ballot_sync(kAll, lane < r.groups && above < r.kept);
    if (kCheck && !r.raw && r.kept < r.groups) {
      // the lowest value that stays against the highest that goes; a value is
      // the sum of up to two keys, each within 2^-18 of its score and 2^-24 of
      // itself, and scores are at most a key plus the largest bias
      float lo = (stay >> lane & 1u) ? (float)value : INFINITY;
      float hi = (stay >> lane & 1u) || lane >= r.groups ? -INFINITY : (float)value;
      lo = -warp_max(-lo);
      hi = warp_max(hi);
      float size = fabsf(lo) + fabsf(hi) + 4.0f * in.bias_max, unit = 7.7e-6f;
      if (r.score == LAPSUM_SCORE_IDENTITY) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (l[i] != -INFINITY) m = fmaxf(m, fabsf(l[i]));
        size = 4.0f * (warp_max(m) + in.bias_max);
        unit = 2.4e-7f;
      }
      certain = hi == -INFINITY || lo - hi > unit * size + 1e-37f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      if (e < r.experts && !(stay >> (e / r.size) & 1u)) o[i] = 0;
    }
  }
  mine = -1;
  int next = -1;  // the choice that would follow
  float my_key = 0.0f, next_key = 0.0f;
  const int rounds = kCheck && !r.raw ? r.k + 1 : r.k;
  for (int j = 0; j < rounds; ++j) {
    O best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (o[i] > best) {
        best = o[i];
        at = i;
      }
    const O m = warp_top(best);
    if (m == 0) break;  // nothing left
    const uint32_t e = __reduce_min_sync(kAll, best == m ? (uint32_t)(at * 32 + lane) : kAll);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if ((uint32_t)(i * 32 + lane) == e) o[i] = 0;
    if (lane == j) {
      mine = (int)e;
      my_key = (float)key_of(m);
    }
    if (j == r.k) {
      mine = lane == r.k ? -1 : mine;
      next = (int)e;
      next_key = (float)key_of(m);
    }
  }
  if (kCheck && !r.raw) {
    // neighbours in the order: apart by more than both errors, or truly equal
    const int at = lane < r.k ? mine : -1;
    const float score = at >= 0 ? load_score<kDtype>(in.scores, in.at + at) : 0.0f;
    const float bias = at >= 0 && in.bias ? __ldg(in.bias + at) : 0.0f;
    int e1 = __shfl_down_sync(kAll, at, 1);
    float key1 = __shfl_down_sync(kAll, my_key, 1);
    float score1 = __shfl_down_sync(kAll, score, 1), bias1 = __shfl_down_sync(kAll, bias, 1);
    if (lane == r.k - 1) {
      e1 = next;
      key1 = next_key;
      score1 = next >= 0 ? load_score<kDtype>(in.scores, in.at + next) : 0.0f;
      bias1 = next >= 0 && in.bias ? __ldg(in.bias + next) : 0.0f;
    }
    if (at >= 0 && e1 >= 0 && !(score == score1 && bias == bias1)) {
      float bound = 2.4e-7f * (fabsf(my_key) + fabsf(key1)) + 1e-37f;  // the last: flushed subnormals
      if (r.score != LAPSUM_SCORE_IDENTITY) bound += 7.7e-6f * (fabsf(my_key - bias) + fabsf(key1 - bias1));
      if (!(my_key - key1 > bound)) certain = false;
    }
    certain = __all_sync(kAll, certain);
  }
  return certain;
}

// This lane's scores and biases, -inf where masked (padding included).  False
// when the token holds a NaN or +inf that is not masked.
template <int kDtype, int kPer>
__device__ __forceinline__ bool load_token(const void* scores, int64_t at, const float* bias, int experts,
                                           float (&l)[kPer], float (&b)[kPer]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    l[i] = e < experts ? load_score<kDtype>(scores, at + e) : -INFINITY;
  }
  bool fine = true;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    b[i] = bias && e < experts ? __ldg(bias + e) : 0.0f;
    if (b[i] == -INFINITY) l[i] = -INFINITY;
    if (l[i] != -INFINITY && !(l[i] < INFINITY && b[i] < INFINITY)) fine = false;
  }
  return __all_sync(kAll, fine);
}

// The choice in fp64, for a token whose fp32 keys lie too close.
template <int kDtype, int kPer>
__device__ __noinline__ int choose_again(const Rule& r, const Keys& in) {
  float l[kPer], b[kPer];
  load_token<kDtype, kPer>(in.scores, in.at, in.bias, r.experts, l, b);
  int mine;
  choose<double, kDtype, kPer>(r, in, l, b, mine);
  return mine;
}

// log of the sigmoid, without overflow
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }

template <int kDtype, int kPer>
__global__ void __launch_bounds__(kThreads) k_route_fwd(const RouteFwd a) {
  const int lane = threadIdx.x & 31;
  Rule r;
  r.experts = a.experts;
  r.k = a.k;
  r.score = a.score;
  r.groups = a.groups;
  r.size = a.experts / a.groups;
  r.kept = a.groups_kept;
  r.top = a.group_top;
  r.raw = !a.bias && (a.groups == 1 || a.group_top == 1);
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
    float l[kPer], b[kPer];
    Keys in;
    in.scores = a.scores;
    in.at = t * a.stride;
    in.bias = a.bias;
    const bool fine = load_token<kDtype, kPer>(a.scores, in.at, a.bias, a.experts, l, b);
    int mine = -1;
    float w = 0.0f;
    if (fine) {
      float m = 0.0f;
      if (!r.raw && r.groups > 1 && a.bias) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (l[i] != -INFINITY) m = fmaxf(m, fabsf(b[i]));
        m = warp_max(m);
      }
      in.bias_max = m;
      if (!choose<float, kDtype, kPer>(r, in, l, b, mine)) mine = choose_again<kDtype, kPer>(r, in);
      if (lane >= a.k) mine = -1;
      const float s = mine >= 0 ? load_score<kDtype>(a.scores, in.at + mine) : -INFINITY;
      if (a.renormalize) {
        if (a.score == LAPSUM_SCORE_IDENTITY) {
          const float v = mine >= 0 ? s : 0.0f;
          const float total = warp_sum(v);
          w = total != 0.0f ? a.scale * v / total : 0.0f;
        } else {  // softmax over the chosen of log s: no sum can vanish
          const float v = a.score == LAPSUM_SCORE_SIGMOID && mine >= 0 ? log_sigmoid(s) : s;
          const float top = warp_max(v);
          const float p = mine >= 0 ? expf(v - top) : 0.0f;
          const float total = warp_sum(p);
          w = mine >= 0 ? a.scale * p / total : 0.0f;
        }
      } else if (a.score == LAPSUM_SCORE_SOFTMAX) {
        float top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) top = fmaxf(top, l[i]);
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (l[i] != -INFINITY) total += expf(l[i] - top);
        total = warp_sum(total);
        w = mine >= 0 ? a.scale * expf(s - top) / total : 0.0f;
      } else if (mine >= 0) {
        w = a.scale * (a.score == LAPSUM_SCORE_SIGMOID ? 1.0f / (1.0f + expf(-s)) : s);
      }
    } else {
      w = __int_as_float(0x7fc00000);
    }
    if (lane < a.k) {
      a.chosen[t * a.k + lane] = mine;
      a.weights[t * a.k + lane] = w;
    }
  }
}

// With g = dL/dw and p the chosen scores:
//   renormalised   dL/dlog s_j = w_j (g_j - sum g w / scale); softmax: dl = that,
//                  sigmoid: times 1 - s_j; identity: (scale g_j - sum g w) / sum s
//   plain          softmax: dl_i = s_i (scale g_i [i chosen] - sum g w), over all
//                  experts; sigmoid: scale g s (1 - s); identity: scale g
template <int kDtype, int kPer>
__global__ void __launch_bounds__(kThreads) k_route_bwd(const RouteBwd a) {
  const int lane = threadIdx.x & 31;
  const bool dense = a.score == LAPSUM_SCORE_SOFTMAX && !a.renormalize;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
    const int64_t at = t * a.stride, out = t * a.grad_stride;
    int e = -1;
    float w = 0.0f, g = 0.0f;
    bool bad = false;
    if (lane < a.k) {
      e = __ldg(a.chosen + t * a.k + lane);
      w = __ldg(a.weights + t * a.k + lane);
      if ((unsigned)e >= (unsigned)a.experts) {
        bad = w != w;
        e = -1;
        w = 0.0f;
      } else {
        g = __ldg(a.grad_weights + t * a.k + lane);
      }
    }
    bad = __any_sync(kAll, bad);
    const float gw = warp_sum(g * w);
    const float s = e >= 0 ? load_score<kDtype>(a.scores, at + e) : 0.0f;
    float d = 0.0f;
    if (a.score == LAPSUM_SCORE_IDENTITY) {
      if (a.renormalize) {
        const float total = warp_sum(e >= 0 ? s : 0.0f);
        d = total != 0.0f ? (a.scale * g - gw) / total : 0.0f;
      } else {
        d = a.scale * g;
      }
    } else if (a.renormalize) {
      d = w * (g - gw / a.scale);
      if (a.score == LAPSUM_SCORE_SIGMOID) d *= 1.0f / (1.0f + expf(s));
    } else if (a.score == LAPSUM_SCORE_SIGMOID) {
      d = g * w / (1.0f + expf(s));
    } else {
      d = w * (g - gw / a.scale);  // s_j (scale g_j - sum g w), s_j = w_j / scale
    }
    float fill = bad ? __int_as_float(0x7fc00000) : 0.0f;
    if (dense && !bad) {
      float l[kPer], b[kPer], top = -INFINITY, total = 0.0f;
      load_token<kDtype, kPer>(a.scores, at, a.bias, a.experts, l, b);
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, l[i]);
      top = warp_max(top);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        l[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - top);
        total += l[i];
      }
      total = warp_sum(total);
      const float by = total > 0.0f ? -gw / total : 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * 32 + lane < a.experts) store_score<kDtype>(a.grad, out + i * 32 + lane, l[i] * by);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * 32 + lane < a.experts) store_score<kDtype>(a.grad, out + i * 32 + lane, fill);
    }
    __syncwarp();  // the chosen experts' gradients replace what stands there
    if (e >= 0 && !bad) store_score<kDtype>(a.grad, out + e, d);
    __syncwarp();
  }
}

template <int kDtype, int kPer>
void fwd_as(const RouteFwd& a, unsigned grid, cudaStream_t st) {
  k_route_fwd<kDtype, kPer><<<grid, kThreads, 0, st>>>(a);
}
template <int kDtype, int kPer>
void bwd_as(const RouteBwd& a, unsigned grid, cudaStream_t st) {
  k_route_bwd<kDtype, kPer><<<grid, kThreads, 0, st>>>(a);
}

#define LAPSUM_BY_EXPERTS(fn, dt, ...)             \
  do {                                             \
    if (a.experts <= 32) fn<dt, 1>(__VA_ARGS__);   \
    else if (a.experts <= 64) fn<dt, 2>(__VA_ARGS__);   \
    else if (a.experts <= 128) fn<dt, 4>(__VA_ARGS__);  \
    else if (a.experts <= 256) fn<dt, 8>(__VA_ARGS__);  \
    else if (a.experts <= 512) fn<dt, 16>(__VA_ARGS__); \
    else fn<dt, 32>(__VA_ARGS__);                  \
  } while (0)
#define LAPSUM_BY_TYPE(fn, ...)                                                        \
  do {                                                                                 \
    if (a.dtype == LAPSUM_F32) LAPSUM_BY_EXPERTS(fn, LAPSUM_F32, __VA_ARGS__);         \
    else if (a.dtype == LAPSUM_BF16) LAPSUM_BY_EXPERTS(fn, LAPSUM_BF16, __VA_ARGS__);  \
    else LAPSUM_BY_EXPERTS(fn, LAPSUM_F16, __VA_ARGS__);                               \
  } while (0)

unsigned blocks_for(int64_t tokens) {
  return (unsigned)std::min<int64_t>((tokens + kWarps - 1) / kWarps, 1 << 20);
}

}  // namespace

cudaError_t launch_route_fwd(const RouteFwd& a, cudaStream_t st) {
  const unsigned grid = blocks_for(a.tokens);
  Launch guard("k_route_fwd", st);
  LAPSUM_BY_TYPE(fwd_as, a, grid, st);
  return cudaGetLastError();
}

cudaError_t launch_route_bwd(const RouteBwd& a, cudaStream_t st) {
  const unsigned grid = blocks_for(a.tokens);
  Launch guard("k_route_bwd", st);
  LAPSUM_BY_TYPE(bwd_as, a, grid, st);
  return cudaGetLastError();
}

}  // namespace lapsum
