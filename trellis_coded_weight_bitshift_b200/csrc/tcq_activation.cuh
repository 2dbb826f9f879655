// Activations of the gated feed-forward block and their slopes, in fp32.
#pragma once

#include "tcq_device.cuh"

namespace tcq {

// 1 / (1 + e^-v): the exponential overflows to infinity for v < -88, whose
// reciprocal is the right 0.
__device__ __forceinline__ float logistic(float v) { return rcp(1.0f + ex2(-1.44269504f * v)); }

// Value and slope of the activation at v.  The tanh form of gelu is
// v * logistic(z), z = 2 sqrt(2/pi) (v + 0.044715 v^3).
__device__ __forceinline__ void activation_slope(float v, int act, float &a, float &d) {
  if (act == TCQ_ACT_SILU) {
    const float p = logistic(v);
    a = v * p;
    d = p + a * logistic(-v);
  } else if (act == TCQ_ACT_GELU) {
    const float p = 0.5f * erfcf(-0.70710678f * v);
    a = v * p;
    d = p + 0.39894228f * v * ex2(-0.72134752f * v * v);
  } else if (act == TCQ_ACT_GELU_TANH) {
    const float vv = fminf(v * v, 1e30f);             // an infinite square would meet a zero below
    const float z = 1.59576912f * v * (1.0f + 0.044715f * vv);
    const float p = logistic(z);
    a = v * p;
    d = p + a * logistic(-z) * 1.59576912f * (1.0f + 0.134145f * vv);
  } else {
    a = v < 0.0f ? 0.0f : v;                          // a NaN stays
    d = v > 0.0f ? 1.0f : 0.0f;
  }
}

template <int ACT>
__device__ __forceinline__ float activation(float v) {
  if (ACT == TCQ_ACT_SILU) return v * logistic(v);
  if (ACT == TCQ_ACT_GELU) return 0.5f * v * erfcf(-0.70710678f * v);
  if (ACT == TCQ_ACT_GELU_TANH) return v * logistic(1.59576912f * v * (1.0f + 0.044715f * v * v));
  return v < 0.0f ? 0.0f : v;
}

// g = act(g) * u, N values.  One branch for all of them: a branch for each value
// made the epilogue the slower half of the kernel (8-bit block 2048 x 2048 x 8192
// with the tanh form: 74.5 us a pass, 60.5 so).
template <int ACT, int N>
__device__ __forceinline__ void gate_as(float (&g)[N], const float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) g[i] = activation<ACT>(g[i]) * u[i];
}
template <int N>
__device__ __forceinline__ void gate(float (&g)[N], const float (&u)[N], int act) {
  if (act == TCQ_ACT_SILU) gate_as<TCQ_ACT_SILU>(g, u);
  else if (act == TCQ_ACT_GELU) gate_as<TCQ_ACT_GELU>(g, u);
  else if (act == TCQ_ACT_GELU_TANH) gate_as<TCQ_ACT_GELU_TANH>(g, u);
  else gate_as<TCQ_ACT_RELU>(g, u);
}

}  // namespace tcq
