// Activations of the gated activation and of the product's epilogue.
#pragma once

#include <hip/hip_runtime.h>

namespace spax {
namespace elem {

// act(g) * up.  With h = exp(-|u| / 2), 1 / (1 + exp(-u)) is 1 / (1 + h h) above zero and
// h h / (1 + h h) below, where one h goes to each factor: exp(-u) itself overflows at u = -88, where act(g)
// is still 2^-121, and h h alone ends there.  1 + h h is in [1, 2], where the hardware's reciprocal
// is good to 2^-23 of itself.
__device__ inline float act_mul(float g, float up, bool gelu) {
  float u = g;
  if (gelu) {
    constexpr float kTwoRootTwoOverPi = 1.59576912160573071176f;
    u = kTwoRootTwoOverPi * (g + 0.044715f * g * g * g);
  }
  const float h = expf(-0.5f * fabsf(u)), f = u < 0.0f ? h : 1.0f;
  return g * f * __builtin_amdgcn_rcpf(1.0f + h * h) * (up * f);
}

}  // namespace elem
}  // namespace spax
