// activation.cuh -- the activations of the experts' products and their
// derivatives, in fp32 for results of 16 bits.
#pragma once

#include <cuda_runtime.h>

#include "lapsum_experts.h"

namespace lapsum {

__device__ __forceinline__ float sigmoid_of(float h) { return __fdividef(1.0f, 1.0f + __expf(-h)); }

// The normal CDF by the rational approximation 7.1.26 of Abramowitz & Stegun
// (|error| of erf <= 1.5e-7): 0.5 erfc(|h| / sqrt 2) = t P(t) exp(-h^2/2) / 2
// with t = 1 / (1 + 0.3275911 |h| / sqrt 2).  The lower tail is not a
// difference.  `e` receives exp(-h^2/2).  A third of erff's instructions: with
// erff the gradient's pass over 16384 x 4096 values was bound by them (167 us).
__device__ __forceinline__ float normal_cdf(float h, float& e) {
  const float t = __fdividef(1.0f, fmaf(0.23164189f, fabsf(h), 1.0f));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  e = __expf(-0.5f * h * h);
  const float q = 0.5f * p * t * e;
  return h < 0.0f ? q : 1.0f - q;
}

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == LAPSUM_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < N; ++c) v[c] = v[c] < 0.0f ? 0.0f : v[c];  // keeps NaN
  } else if (act == LAPSUM_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < N; ++c) v[c] *= sigmoid_of(v[c]);
  } else if (act == LAPSUM_ACT_GELU) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      float e;
      v[c] *= normal_cdf(v[c], e);
    }
  }
}

// g = g * act'(h)
template <int N>
__device__ __forceinline__ void differentiate(float (&g)[N], const float (&h)[N], int act) {
  if (act == LAPSUM_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < N; ++c) g[c] = h[c] <= 0.0f ? 0.0f : g[c];
  } else if (act == LAPSUM_ACT_SILU) {  // s (1 + h (1 - s))
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float s = sigmoid_of(h[c]);
      g[c] *= s * fmaf(h[c], 1.0f - s, 1.0f);
    }
  } else if (act == LAPSUM_ACT_GELU) {  // Phi(h) + h phi(h)
#pragma unroll
    for (int c = 0; c < N; ++c) {
      float e;
      const float cdf = normal_cdf(h[c], e);
      g[c] *= fmaf(0.39894228f * h[c], e, cdf);
    }
  }
}

}  // namespace lapsum
