// route.cu -- the choice of experts and its gradient.
//
// One warp per token: lane l holds kPer neighbours, experts kPer l .. ; a choice
// is one integer maximum over the warp (keys mapped to integers of the same
// order) and the lowest lane that has it.  Groups that are whole lanes, a power
// of two of them, find their two highest keys in log2 steps, all groups at
// once.  The floor is the scores' bytes; what bounds it is the issue of the k
// rounds, some 40 instructions each.
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

// of the keys: the fp32 forms are the fast ones, whose error the bounds below cover
__device__ __forceinline__ float exp_of(float v) { return __expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float quotient(float a, float b) { return __fdividef(a, b); }
__device__ __forceinline__ double quotient(double a, double b) { return a / b; }

struct Rule {
  int experts, k, score;
  int groups, size, kept, top;  // size: experts of a group
  int lanes;                    // of a group: a power of two, or 0 (groups are not whole lanes)
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

// (a, b) = the two highest of a >= b and c >= d
template <typename O>
__device__ __forceinline__ void top_two(O& a, O& b, O c, O d) {
  b = max(min(a, c), max(b, d));
  a = max(a, c);
}
template <typename O>
__device__ __forceinline__ O shuffle_xor(O v, int d) {
  return (O)__shfl_xor_sync(kAll, (unsigned long long)v, d);
}
template <>
__device__ __forceinline__ uint32_t shuffle_xor<uint32_t>(uint32_t v, int d) {
  return __shfl_xor_sync(kAll, v, d);
}

// Lane j < k gets the token's j-th choice (or -1).  l: this lane's scores, -inf
// where masked; b: its biases.  picked: k + 1 pairs (expert, key) in shared
// memory.  Returns whether the choice is certain at the precision of K (always,
// for fp64 and for raw keys).
template <typename K, int kDtype, int kPer>
__device__ __forceinline__ bool choose(const Rule& r, const Keys& in, const float (&l)[kPer], const float (&b)[kPer],
                                       int2* picked, int& mine) {
  using O = typename Order<K>::O;
  constexpr bool kCheck = sizeof(K) == 4;
  const int lane = threadIdx.x & 31;
  O o[kPer];
  bool certain = true;
  if (r.raw) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = l[i] == -INFINITY ? O(0) : ordered((K)l[i]);
  } else {
    K top = 0, scale = 1;
    if (r.score == LAPSUM_SCORE_SOFTMAX) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = fmaxf(m, l[i]);
      top = (K)warp_max(m);
      K s = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (l[i] != -INFINITY) s += exp_of((K)l[i] - top);
      scale = quotient((K)1, warp_sum(s));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      K s = (K)l[i];
      if (r.score == LAPSUM_SCORE_SOFTMAX) s = exp_of(s - top) * scale;
      if (r.score == LAPSUM_SCORE_SIGMOID) s = quotient((K)1, (K)1 + exp_of(-s));
      o[i] = l[i] == -INFINITY ? O(0) : ordered(s + (K)b[i]);
    }
  }
  if (r.kept < r.groups) {
    // the value of group g: in all its lanes, or in lane g where they are not whole
    O first = 0, second = 0;
    int g = lane, lanes = 1;
    if (r.lanes) {
      lanes = r.lanes;
      g = lane / lanes;
#pragma unroll
      for (int i = 0; i < kPer; ++i) top_two(first, second, o[i], O(0));
      for (int d = 1; d < lanes; d <<= 1) {
        const O c = shuffle_xor(first, d), e = shuffle_xor(second, d);
        top_two(first, second, c, e);
      }
    } else {
      for (int q = 0; q < r.groups; ++q) {
        const int e0 = q * r.size - lane * kPer, e1 = e0 + r.size;
        O c = 0, e = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i >= e0 && i < e1) top_two(c, e, o[i], O(0));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const O x = shuffle_xor(c, d), y = shuffle_xor(e, d);
          top_two(c, e, x, y);
        }
        if (lane == q) {
          first = c;
          second = e;
        }
      }
    }
    K value = first ? key_of(first) : (K)-INFINITY;
    if (r.top == 2 && second) value += key_of(second);
    if (g >= r.groups) value = -INFINITY;
    int above = 0;
    for (int q = 0; q < r.groups; ++q) {
      const K v = __shfl_sync(kAll, value, q * lanes);
      above += (v > value || (v == value && q < g)) ? 1 : 0;
    }
    const bool stays = g < r.groups && above < r.kept;
    if (kCheck && !r.raw) {
      // the lowest value that stays against the highest that goes; a value is
      // the sum of up to two keys, each within 2^-18 of its score and 2^-24 of
      // itself, and scores are at most a key plus the largest bias
      const float lo = -warp_max(stays ? -(float)value : -INFINITY);
      const float hi = warp_max(stays || g >= r.groups ? -INFINITY : (float)value);
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
    if (r.lanes) {
      if (!stays) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = 0;
      }
    } else {
      const uint32_t stay = __ballot_sync(kAll, stays);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane * kPer + i;
        if (e < r.experts && !(stay >> (e / r.size) & 1u)) o[i] = 0;
      }
    }
  }
  const int rounds = kCheck && !r.raw ? r.k + 1 : r.k;  // with the choice that would follow
  if (lane < rounds || lane == 0) picked[lane] = make_int2(-1, 0);
  if (lane == 0) picked[r.k] = make_int2(-1, 0);
  __syncwarp();
  for (int j = 0; j < rounds; ++j) {
    O best = o[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, o[i]);
    const O m = warp_top(best);
    if (m == 0) break;  // nothing left
    if (lane == __ffs(__ballot_sync(kAll, best == m)) - 1) {
      int at = 0;
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i)
        if (o[i] == m) at = i;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == at) o[i] = 0;
      picked[j] = make_int2(lane * kPer + at, __float_as_int((float)key_of(m)));
    }
  }
  __syncwarp();
  mine = lane < r.k ? picked[lane].x : -1;
  if (kCheck && !r.raw) {
    // neighbours in the order: apart by more than both errors, or truly equal
    if (mine >= 0) {
      const int e1 = picked[lane + 1].x;
      if (e1 >= 0) {
        const float key = __int_as_float(picked[lane].y), key1 = __int_as_float(picked[lane + 1].y);
        const float score = load_score<kDtype>(in.scores, in.at + mine), score1 = load_score<kDtype>(in.scores, in.at + e1);
        const float bias = in.bias ? __ldg(in.bias + mine) : 0.0f, bias1 = in.bias ? __ldg(in.bias + e1) : 0.0f;
        float bound = 2.4e-7f * (fabsf(key) + fabsf(key1)) + 1e-37f;  // the last: flushed subnormals
        if (r.score != LAPSUM_SCORE_IDENTITY) bound += 7.7e-6f * (fabsf(key - bias) + fabsf(key1 - bias1));
        if (!(score == score1 && bias == bias1) && !(key - key1 > bound)) certain = false;
      }
    }
    certain = __all_sync(kAll, certain);
  }
  __syncwarp();
  return certain;
}

// kPer neighbouring scores; vec: as one access of up to 16 bytes each
template <int kDtype, int kPer>
__device__ __forceinline__ void load_scores(const void* scores, int64_t at, int n, bool vec, float (&l)[kPer]) {
  constexpr int kSize = kDtype == LAPSUM_F32 ? 4 : 2;
  constexpr int kBytes = kPer * kSize < 16 ? kPer * kSize : 16, kEach = kBytes / kSize;
  if (vec && kBytes > 4) {
    if (n > 0) {
#pragma unroll
      for (int q = 0; q < kPer / kEach; ++q) {
        uint32_t w[4];
        const char* p = static_cast<const char*>(scores) + (at + q * kEach) * kSize;
        if (kBytes == 16) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
          w[0] = v.x, w[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const uint32_t u = kSize == 4 ? w[i % 4] : (w[i / 2 % 4] >> (16 * (i & 1)) & 0xffffu);
          l[q * kEach + i] = kDtype == LAPSUM_F32 ? __uint_as_float(u)
                             : kDtype == LAPSUM_BF16 ? __uint_as_float(u << 16)
                                                     : __half2float(__ushort_as_half((uint16_t)u));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) l[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) l[i] = i < n ? load_score<kDtype>(scores, at + i) : -INFINITY;
  }
}

template <int kDtype, int kPer>
__device__ __forceinline__ void store_scores(void* grad, int64_t at, int n, bool vec, const float (&v)[kPer]) {
  constexpr int kSize = kDtype == LAPSUM_F32 ? 4 : 2;
  constexpr int kBytes = kPer * kSize < 16 ? kPer * kSize : 16, kEach = kBytes / kSize;
  if (vec && kBytes > 4) {
    if (n > 0) {
#pragma unroll
      for (int q = 0; q < kPer / kEach; ++q) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float f = v[q * kEach + i];
          if (kSize == 4)
            w[i % 4] = __float_as_uint(f);
          else
            w[i / 2 % 4] |= (uint32_t)(kDtype == LAPSUM_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f))
                                                             : __half_as_ushort(__float2half_rn(f)))
                            << (16 * (i & 1));
        }
        char* p = static_cast<char*>(grad) + (at + q * kEach) * kSize;
        if (kBytes == 16)
          *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
          *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) store_score<kDtype>(grad, at + i, v[i]);
  }
}

// This lane's scores and biases, -inf where masked (padding included).  False
// when the token holds a NaN or +inf that is not masked.
template <int kDtype, int kPer>
__device__ __forceinline__ bool load_token(const void* scores, int64_t at, const float* bias, int experts, bool vec,
                                           float (&l)[kPer], float (&b)[kPer]) {
  const int lane = threadIdx.x & 31, e0 = lane * kPer, n = max(0, min(kPer, experts - e0));
  load_scores<kDtype, kPer>(scores, at + e0, n, vec, l);
  bool fine = true;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    b[i] = bias && i < n ? __ldg(bias + e0 + i) : 0.0f;
    if (b[i] == -INFINITY) l[i] = -INFINITY;
    if (l[i] != -INFINITY && !(l[i] < INFINITY && b[i] < INFINITY)) fine = false;
  }
  return __all_sync(kAll, fine);
}

// The choice in fp64, for a token whose fp32 keys lie too close.
template <int kDtype, int kPer>
__device__ __noinline__ int choose_again(const Rule& r, const Keys& in, int2* picked) {
  float l[kPer], b[kPer];
  load_token<kDtype, kPer>(in.scores, in.at, in.bias, r.experts, false, l, b);
  int mine;
  choose<double, kDtype, kPer>(r, in, l, b, picked, mine);
  return mine;
}

// log of the sigmoid, without overflow
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }

template <int kDtype, int kPer>
__global__ void __launch_bounds__(kThreads) k_route_fwd(const RouteFwd a) {
  __shared__ int2 all_picked[kWarps][LAPSUM_EXPERTS_MAX_K + 1];
  int2* picked = all_picked[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  Rule r;
  r.experts = a.experts;
  r.k = a.k;
  r.score = a.score;
  r.groups = a.groups;
  r.size = a.experts / a.groups;
  r.kept = a.groups_kept;
  r.top = a.group_top;
  r.raw = !a.bias && (a.groups_kept == a.groups || a.group_top == 1);
  r.lanes = r.size % kPer == 0 && ((r.size / kPer) & (r.size / kPer - 1)) == 0 ? r.size / kPer : 0;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
    float l[kPer], b[kPer];
    Keys in;
    in.scores = a.scores;
    in.at = t * a.stride;
    in.bias = a.bias;
    const bool fine = load_token<kDtype, kPer>(a.scores, in.at, a.bias, a.experts, a.vec, l, b);
    int mine = -1;
    float w = 0.0f;
    if (fine) {
      float m = 0.0f;
      if (!r.raw && r.kept < r.groups && a.bias) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (l[i] != -INFINITY) m = fmaxf(m, fabsf(b[i]));
        m = warp_max(m);
      }
      in.bias_max = m;
      if (!choose<float, kDtype, kPer>(r, in, l, b, picked, mine)) mine = choose_again<kDtype, kPer>(r, in, picked);
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
          if (l[i] != -INFINITY) total += __expf(l[i] - top);
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
    float v[kPer];
    const int e0 = lane * kPer, n = max(0, min(kPer, a.experts - e0));
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = bad ? __int_as_float(0x7fc00000) : 0.0f;
    if (dense && !bad) {
      float b[kPer], top = -INFINITY, total = 0.0f;
      load_token<kDtype, kPer>(a.scores, at, a.bias, a.experts, a.vec, v, b);
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, v[i]);
      top = warp_max(top);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = v[i] == -INFINITY ? 0.0f : __expf(v[i] - top);
        total += v[i];
      }
      total = warp_sum(total);
      const float by = total > 0.0f ? -gw / total : 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] *= by;
    }
    store_scores<kDtype, kPer>(a.grad, out + e0, n, a.grad_vec, v);
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

// every lane's scores are whole and start on a boundary of their bytes (16 at most)
bool whole_lanes(const void* p, int64_t stride, int dtype, int experts) {
  int per = 1;
  while (per * 32 < experts) per *= 2;
  const int size = dtype == LAPSUM_F32 ? 4 : 2, bytes = std::min(16, per * size);
  return experts % per == 0 && (uintptr_t)p % bytes == 0 && stride * size % bytes == 0;
}

unsigned blocks_for(int64_t tokens) {
  return (unsigned)std::min<int64_t>((tokens + kWarps - 1) / kWarps, 1 << 20);
}

}  // namespace

cudaError_t launch_route_fwd(RouteFwd a, cudaStream_t st) {
  a.vec = whole_lanes(a.scores, a.stride, a.dtype, a.experts);
  const unsigned grid = blocks_for(a.tokens);
  Launch guard("k_route_fwd", st);
  LAPSUM_BY_TYPE(fwd_as, a, grid, st);
  return cudaGetLastError();
}

cudaError_t launch_route_bwd(RouteBwd a, cudaStream_t st) {
  a.vec = whole_lanes(a.scores, a.stride, a.dtype, a.experts);
  a.grad_vec = whole_lanes(a.grad, a.grad_stride, a.dtype, a.experts);
  const unsigned grid = blocks_for(a.tokens);
  Launch guard("k_route_bwd", st);
  LAPSUM_BY_TYPE(bwd_as, a, grid, st);
  return cudaGetLastError();
}

}  // namespace lapsum
