// Activations of the fused products and their derivatives, in fp32.
#pragma once

#include "common.hpp"

// logistic function with the hardware's exp2 and reciprocal (about 2 ulp)
__device__ __forceinline__ float act_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

#define ACT_GELU_C 0.7978845608028654f   // sqrt(2 / pi)
#define ACT_GELU_Q 0.044715f

// gelu is z Phi(z) with Phi(z) = erfc(-z / sqrt 2) / 2, which keeps its
// relative precision for negative z; its tanh form is z s(2 u), u = c (z + q
// z^3), since (1 + tanh u) / 2 = s(2 u).
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;   // (a NaN stays one)
    case MOE_ACT_SILU: return z * act_sigmoid(z);
    case MOE_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case MOE_ACT_GELU_TANH:
      return z * act_sigmoid(2.0f * ACT_GELU_C * (z + ACT_GELU_Q * z * z * z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : (z != z ? z : 0.f);
    case MOE_ACT_SILU: {
      const float s = act_sigmoid(z);
      return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU:
      return 0.5f * erfcf(-0.70710678118654752f * z) +
             0.3989422804014327f * z * __expf(-0.5f * z * z);
    case MOE_ACT_GELU_TANH: {
      if (fabsf(z) > 30.f) return z > 0.f ? 1.f : 0.f;   // its limits, ahead of z^2's overflow
      const float s = act_sigmoid(2.0f * ACT_GELU_C * (z + ACT_GELU_Q * z * z * z));
      return s + z * s * (1.0f - s) * 2.0f * ACT_GELU_C * (1.0f + 3.0f * ACT_GELU_Q * z * z);
    }
    default: return 1.0f;
  }
}
