// The gated block's activations (qlora_activation), on the device.
#pragma once

#include "common.h"

namespace qlora {

// silu  g s,  s = 1 / (1 + e^-g);  gelu (tanh form)  g / (1 + e^-2t),  t = sqrt(2/pi) (g + 0.044715 g^3):
// (1 + tanh t) / 2 is the logistic function of 2t, so both are g times one, and take one exponential.
__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}
constexpr float kGeluA = 2.0f * 0.7978845608028654f, kGeluB = 0.044715f;

__device__ __forceinline__ float activate(float g, int act) {
  const float x = act == 0 ? g : kGeluA * g * __builtin_fmaf(kGeluB * g, g, 1.0f);
  return g * logistic(x);
}

// the value, and the derivative  s + g s (1 - s) x'(g)
__device__ __forceinline__ float activate(float g, int act, float& slope) {
  const float x = act == 0 ? g : kGeluA * g * __builtin_fmaf(kGeluB * g, g, 1.0f);
  // (past 10^4 the factor s (1 - s) is 0, and x' may not be infinite beside it)
  const float gc = __builtin_fminf(__builtin_fabsf(g), 1e4f);
  const float dx = act == 0 ? 1.0f : kGeluA * __builtin_fmaf(3.0f * kGeluB * gc, gc, 1.0f);
  const float s = logistic(x);
  slope = __builtin_fmaf(g * s * (1.0f - s), dx, s);
  return g * s;
}

}  // namespace qlora
