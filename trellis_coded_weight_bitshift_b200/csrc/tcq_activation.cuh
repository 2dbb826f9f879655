// Activations of the gated feed-forward block and their slopes, in fp32.
#pragma once

#include "tcq_device.cuh"

namespace tcq {

// 1 / (1 + e^-v): the exponential overflows to infinity for v < -88, whose
// reciprocal is the right 0.
__device__ __forceinline__ float logistic(float v) { return rcp(1.0f + ex2(-1.44269504f * v)); }

// The normal distribution's density z and distribution function p at v.  For v >= 0
// 1 - p = e^(-v^2 / 2) t P(t), t = 1 / (1 + 0.3 v), with P of degree 7 fitted to the least
// largest relative error on [0, 14] by reweighted least squares (1.5e-7), so that the tail
// is right to its own digits: it is what gelu is for v < 0.  With the roundings, of the
// exponent most of all, the relative error is within (8 + 3/4 v^2) 2^-23 (3e-6 measured at
// -8).  A five-term form with an absolute bound (7.5e-8) left 5e-5 at -3 and 1e-2 at -8.
// Two special-function instructions and eleven others, where erfc takes about forty (8-bit
// gated block 2048 x 2048 x 8192: 62.4 us so, 61.4 with the five-term form, 76 with erfc).
__host__ __device__ constexpr float tail_term(int i) {
  constexpr float c[8] = {0.119629301f,   0.120753959f, 0.0999134481f, 0.12856181f,
                          -0.0536840446f, 0.206354007f, -0.157203421f, 0.0356748663f};
  return c[i];
}
constexpr float kTailRate = 0.3f;
__device__ __forceinline__ void normal(float v, float &z, float &p) {
  const float e = ex2(-0.72134752f * v * v), t = rcp(fmaf(fabsf(v), kTailRate, 1.0f));
  z = 0.39894228f * e;
  float q = tail_term(7);
#pragma unroll
  for (int i = 6; i >= 0; --i) q = fmaf(q, t, tail_term(i));
  q *= t * e;
  p = v < 0.0f ? q : 1.0f - q;
}

// Value and slope of the activation at v.  The tanh form of gelu is
// v * logistic(z), z = 2 sqrt(2/pi) (v + 0.044715 v^3).
__device__ __forceinline__ void activation_slope(float v, int act, float &a, float &d) {
  if (act == TCQ_ACT_SILU) {
    const float p = logistic(v);
    a = v * p;
    d = p + a * logistic(-v);
  } else if (act == TCQ_ACT_GELU) {
    float z, p;
    normal(v, z, p);
    a = v * p;
    d = p + v * z;
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

// The activation of two values at once, times u: pairs where the hardware has them.
template <int ACT>
__device__ __forceinline__ f2_t gated_pair(f2_t g, f2_t u) {
  if (ACT == TCQ_ACT_SILU || ACT == TCQ_ACT_GELU_TANH) {
    // g * logistic(z), z = g or 2 sqrt(2/pi) (g + 0.044715 g^3); t = -z log2(e)
    f2_t t;
    if (ACT == TCQ_ACT_SILU) {
      t = f2mul(g, f2(-1.44269504f, -1.44269504f));
    } else {
      const f2_t w = f2fma(f2mul(g, g), f2(-0.10294324f, -0.10294324f), f2(-2.30220820f, -2.30220820f));
      t = f2mul(g, w);
    }
    const f2_t d = f2add(f2(ex2(f2lo(t)), ex2(f2hi(t))), f2(1.0f, 1.0f));
    return f2mul(f2mul(g, f2(rcp(f2lo(d)), rcp(f2hi(d)))), u);
  }
  if (ACT == TCQ_ACT_GELU) {
    const f2_t e = f2mul(f2mul(g, g), f2(-0.72134752f, -0.72134752f));
    const f2_t d = f2fma(f2(fabsf(f2lo(g)), fabsf(f2hi(g))), f2(kTailRate, kTailRate), f2(1.0f, 1.0f));
    const f2_t t = f2(rcp(f2lo(d)), rcp(f2hi(d)));
    f2_t q = f2(tail_term(7), tail_term(7));
#pragma unroll
    for (int i = 6; i >= 0; --i) q = f2fma(q, t, f2(tail_term(i), tail_term(i)));
    q = f2mul(q, f2mul(t, f2(ex2(f2lo(e)), ex2(f2hi(e)))));
    const float lo = f2lo(g) < 0.0f ? f2lo(q) : 1.0f - f2lo(q), hi = f2hi(g) < 0.0f ? f2hi(q) : 1.0f - f2hi(q);
    return f2mul(f2mul(g, f2(lo, hi)), u);
  }
  return f2mul(f2(f2lo(g) < 0.0f ? 0.0f : f2lo(g), f2hi(g) < 0.0f ? 0.0f : f2hi(g)), u);
}

// g = act(g) * u, N values.  One branch for all of them: a branch for each value
// made the epilogue the slower half of the kernel (8-bit block 2048 x 2048 x 8192
// with the tanh form: 74.5 us a pass, 60.5 so).
template <int ACT, int N>
__device__ __forceinline__ void gate_as(float (&g)[N], const float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const f2_t r = gated_pair<ACT>(f2(g[i], g[i + 1]), f2(u[i], u[i + 1]));
    g[i] = f2lo(r);
    g[i + 1] = f2hi(r);
  }
}
template <int N>
__device__ __forceinline__ void gate(float (&g)[N], const float (&u)[N], int act) {
  if (act == TCQ_ACT_SILU) gate_as<TCQ_ACT_SILU>(g, u);
  else if (act == TCQ_ACT_GELU) gate_as<TCQ_ACT_GELU>(g, u);
  else if (act == TCQ_ACT_GELU_TANH) gate_as<TCQ_ACT_GELU_TANH>(g, u);
  else gate_as<TCQ_ACT_RELU>(g, u);
}

}  // namespace tcq
