// Activations of gated blocks and their slopes, in fp32.
#pragma once

#include "common.cuh"

namespace moe {

// 1 / (1 + exp(-v)); 0 where the sum is above 2^126, a value below 2^-126.
__device__ __forceinline__ float sigmoid(float v) {
  return __fdividef(1.0f, 1.0f + __expf(-v));
}

// 0.5 (1 + tanh(u)) = sigmoid(2 u) of u = sqrt(2 / pi) (g + 0.044715 g^3).
__device__ __forceinline__ float gelu_inner(float g) {
  return 0.7978845608f * g * fmaf(0.044715f * g, g, 1.0f);
}

__device__ __forceinline__ float act_value(int act, float g) {
  if (act == MOE_ACT_SILU) return g * sigmoid(g);
  // beyond 16 the sigmoid is 0 or 1 in fp32, and the cube need not be finite
  return g * sigmoid(2.0f * gelu_inner(fminf(fmaxf(g, -16.0f), 16.0f)));
}

// Value and slope.
__device__ __forceinline__ float2 act_slope(int act, float g) {
  if (act == MOE_ACT_SILU) {
    const float s = sigmoid(g);
    return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
  }
  const float c = fminf(fmaxf(g, -16.0f), 16.0f);
  const float s = sigmoid(2.0f * gelu_inner(c));
  const float inner = 0.7978845608f * fmaf(3.0f * 0.044715f * c, c, 1.0f);
  return make_float2(g * s, fmaf(2.0f * g * inner, s * (1.0f - s), s));
}

}  // namespace moe
