// activation.cuh -- the activations of the experts' products and their
// derivatives, in fp32 for results of 16 bits.
#pragma once

#include <cuda_runtime.h>

#include "lapsum_experts.h"

namespace lapsum {

__device__ __forceinline__ float sigmoid_of(float h) { return __fdividef(1.0f, 1.0f + __expf(-h)); }

// The normal CDF's lower tail is r(z) exp(-z^2/2), r(z) = 0.5 erfcx(z / sqrt 2); the
// upper one is 1 minus that.  r = t P(t) with t = 1 / (1 + 0.362 z): a minimax fit of its
// relative error on 0 <= z <= 13.5 (least squares in t, the weights follow the error),
// 1.0e-6 in fp32, so that gelu keeps its relative accuracy where it vanishes (the
// exponential adds up to 1.6e-5 of the value at z = 13, 2e-6 at 4).  The exponential
// is the last factor: r times it would underflow before z r times it does.  With erff the
// gradient's pass over 16384 x 4096 values was bound by it (167 us).
__device__ __forceinline__ float lower_tail(float z) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.362f, z, 1.0f)));
  float p = fmaf(t, 0.0480388142f, -0.180348381f);
  p = fmaf(t, p, 0.177071124f);
  p = fmaf(t, p, 0.0285237245f);
  p = fmaf(t, p, 0.139540404f);
  p = fmaf(t, p, 0.14266938f);
  p = fmaf(t, p, 0.144505292f);
  return p * t;
}
// exp(-h^2 / 2)
__device__ __forceinline__ float bell(float h) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h * h * -0.72134752f));
  return e;
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
      // max(h, 0) - |h| r exp(-h^2/2); from 20 on the exponential is 0
      const float z = fminf(fabsf(v[c]), 20.0f);
      v[c] = fmaf(-(z * lower_tail(z)), bell(v[c]), fmaxf(v[c], 0.0f));
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
      const float r = lower_tail(fabsf(h[c]));
      const bool low = h[c] < 0.0f;
      g[c] *= fmaf(bell(h[c]), fmaf(0.39894228f, h[c], low ? r : -r), low ? 0.0f : 1.0f);
    }
  }
}

}  // namespace lapsum
