// Activations of the fused products and their derivatives, in fp32.
#pragma once

#include "common.hpp"

// Logistic function with the hardware's exp2 and reciprocal.  The exp's argument
// is rounded, so the relative error grows with it where the exp counts: of
// negative z silu was off by (3 + |z|) 2^-24 at most over [-87, 0] (of positive
// ones 3 x 2^-24), gelu's tanh form by (4 + 2.8 |2 u|) 2^-24 of its argument
// below, and where the result nears 2^-126 it is 0.
__device__ __forceinline__ float act_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

#define ACT_GELU_C 0.7978845608028654f   // sqrt(2 / pi)
#define ACT_GELU_Q 0.044715f

// Phi(z) with its relative precision for negative z too: Phi(-|z|) = e^(-x^2)
// E(x) / 2 with x = |z| / sqrt 2 and E(x) = e^(x^2) erfc(x), and Phi(z) = 1 -
// Phi(-z).  E is smooth and falls like 1/x, so it is a polynomial in t = 1 / (1
// + 0.39 x); these coefficients are a weighted least-squares fit made minimax in
// the relative error by reweighting (7e-8 on [0, 14]; beyond, the exponential
// is zero).  In fp32 gelu was off by 5.5 x 2^-24 of its value at most for z > 0 and
// by (8 + 0.75 z^2) 2^-24 below, where the exp's rounded argument is most of it.
// gauss: e^(-z^2 / 2), which the slope needs too.  (erfcf took 39 us of the
// epilogue of 8191 x 2048 outputs, this takes 10.)
__device__ __forceinline__ float act_phi(float z, float& gauss) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.39f * 0.70710678118654752f * fabsf(z));
  gauss = __expf(-0.5f * z * z);
  float e = 0.053770684f;
  e = fmaf(e, t, -0.21629582f);
  e = fmaf(e, t, 0.2476963f);
  e = fmaf(e, t, -0.05903618f);
  e = fmaf(e, t, 0.16900781f);
  e = fmaf(e, t, 0.16050708f);
  e = fmaf(e, t, 0.20432884f);
  e = fmaf(e, t, 0.21998748f);
  e = fmaf(e, t, 0.22003388f);
  const float h = 0.5f * gauss * (e * t);
  return z < 0.f ? h : 1.0f - h;
}

// gelu is z Phi(z); its tanh form is z s(2 u), u = c (z + q z^3), since (1 +
// tanh u) / 2 = s(2 u).
// z p for a p that falls to 0 faster than z grows: 0 at z = -infinity too.  (A
// NaN z is passed over by the maximum; p carries it.  Asking for p == 0 instead
// took 2 us more of the epilogue of 8191 x 2048 outputs.)
__device__ __forceinline__ float act_times(float z, float p) {
  return fmaxf(z, -3.402823466e38f) * p;
}

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;   // (a NaN stays one)
    case MOE_ACT_SILU: return act_times(z, act_sigmoid(z));
    case MOE_ACT_GELU: {
      float gauss;
      return act_times(z, act_phi(z, gauss));
    }
    case MOE_ACT_GELU_TANH:
      return act_times(z, act_sigmoid(2.0f * ACT_GELU_C * (z + ACT_GELU_Q * z * z * z)));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : (z != z ? z : 0.f);
    case MOE_ACT_SILU: {
      // (beyond 100 the slope is its limit, and an infinite z would meet a 0; s carries a NaN)
      const float s = act_sigmoid(z), w = fminf(fmaxf(z, -100.f), 100.f);
      return s * (1.0f + w * (1.0f - s));
    }
    case MOE_ACT_GELU: {
      if (fabsf(z) > 30.f) return z > 0.f ? 1.f : 0.f;   // its limits, ahead of infinity times 0
      float gauss;
      const float phi = act_phi(z, gauss);
      return phi + 0.3989422804014327f * z * gauss;
    }
    case MOE_ACT_GELU_TANH: {
      if (fabsf(z) > 30.f) return z > 0.f ? 1.f : 0.f;   // its limits, ahead of z^2's overflow
      const float s = act_sigmoid(2.0f * ACT_GELU_C * (z + ACT_GELU_Q * z * z * z));
      return s + z * s * (1.0f - s) * 2.0f * ACT_GELU_C * (1.0f + 3.0f * ACT_GELU_Q * z * z);
    }
    default: return 1.0f;
  }
}
