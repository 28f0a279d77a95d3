// The gate activations and their derivatives, in fp32.
#pragma once

#include <cuda_runtime.h>

#include "fwt.h"

namespace fwt {
namespace ff {

// 1 / (1 + exp(-z)).  The exponential saturates to 0 or Inf and the quotient to 1 or 0.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// value = act(g), slope = act'(g).
//   silu: g p, p + g p (1 - p), p = logistic(g)
//   gelu: (1 + tanh z) / 2 = logistic(2 z), so the same with p = logistic(c (g + 0.044715 g^3)),
//         c = 2 sqrt(2 / pi), and the inner derivative c (1 + 3 * 0.044715 g^2)
template <int ACT>
__device__ __forceinline__ void activation(float g, float& value, float& slope) {
  if constexpr (ACT == FWT_RELU) {
    value = g > 0.f ? g : (g == g ? 0.f : g);
    slope = g > 0.f ? 1.f : (g == g ? 0.f : g);
  } else {
    constexpr float c = 1.5957691216057308f, c3 = 0.044715f;
    const float p = logistic(ACT == FWT_SILU ? g : c * (g + c3 * g * g * g));
    const float inner = ACT == FWT_SILU ? 1.f : c * (1.f + 3.f * c3 * g * g);
    // far below zero p is 0 while g (and the cube) may be -Inf: the limit is 0
    value = p == 0.f ? 0.f : g * p;
    slope = p + (p == 0.f || p == 1.f ? 0.f : value * (1.f - p) * inner);
  }
}

__device__ __forceinline__ void activate(int act, float g, float& value, float& slope) {
  if (act == FWT_SILU) activation<FWT_SILU>(g, value, slope);
  else if (act == FWT_GELU) activation<FWT_GELU>(g, value, slope);
  else activation<FWT_RELU>(g, value, slope);
}

}  // namespace ff
}  // namespace fwt
