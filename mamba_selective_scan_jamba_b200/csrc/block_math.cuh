// Activations of the decoder block's operators and their derivatives (float32).
#pragma once

#include <cuda_bf16.h>

#include "jmix.h"

namespace jmix {

__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// GELU by erfc, v Phi(v) = v erfc(-v / sqrt 2) / 2: no cancellation for v < 0.
__device__ __forceinline__ float act_apply(float v, int act) {
  switch (act) {
    case JM_ACT_RELU: return v > 0.0f ? v : (v != v ? v : 0.0f);
    case JM_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678f);
    case JM_ACT_SILU: return v / (1.0f + __expf(-v));
    default: return v;
  }
}

__device__ __forceinline__ float act_grad(float v, int act) {
  switch (act) {
    case JM_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
    case JM_ACT_GELU:  // Phi(v) + v phi(v)
      return 0.5f * erfcf(v * -0.70710678f) + v * 0.39894228f * __expf(-0.5f * v * v);
    case JM_ACT_SILU: {
      const float s = 1.0f / (1.0f + __expf(-v));
      return s * (1.0f + v * (1.0f - s));
    }
    default: return 1.0f;
  }
}

}  // namespace jmix
