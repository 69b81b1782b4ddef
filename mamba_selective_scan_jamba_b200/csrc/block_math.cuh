// Activations of the decoder block's operators and their derivatives (float32).
#pragma once

#include <cuda_bf16.h>

#include "jmix.h"

namespace jmix {

__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The normal distribution's Phi(v), and e = exp(-v^2 / 2) for its density: erfc(z) =
// poly(t) t exp(-z^2), t = 1 / (1 + 0.3275911 z), z = |v| / sqrt 2 (Abramowitz and Stegun,
// 7.1.26: within 1.5e-7).  Phi(v) = erfc(z) / 2 for v < 0, so that no difference from 1
// loses the small values.
__device__ __forceinline__ float normal_cdf(float v, float& e) {
  const float t = __fdividef(1.0f, fmaf(fabsf(v), 0.3275911f * 0.70710678f, 1.0f));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  e = __expf(-0.5f * v * v);
  const float half_erfc = 0.5f * p * t * e;
  return v < 0.0f ? half_erfc : 1.0f - half_erfc;
}

__device__ __forceinline__ float act_apply(float v, int act) {
  switch (act) {
    case JM_ACT_RELU: return v > 0.0f ? v : (v != v ? v : 0.0f);
    case JM_ACT_GELU: {
      float e;
      return v * normal_cdf(v, e);
    }
    case JM_ACT_SILU: return v * sigmoid_f(v);
    default: return v;
  }
}

__device__ __forceinline__ float act_grad(float v, int act) {
  switch (act) {
    case JM_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
    case JM_ACT_GELU: {  // Phi(v) + v phi(v)
      float e;
      const float c = normal_cdf(v, e);
      return fmaf(v * 0.39894228f, e, c);
    }
    case JM_ACT_SILU: {
      const float s = sigmoid_f(v);
      return s * fmaf(v, 1.0f - s, 1.0f);
    }
    default: return 1.0f;
  }
}

}  // namespace jmix
