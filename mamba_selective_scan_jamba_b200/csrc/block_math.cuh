// Activations of the decoder block's operators and their derivatives (float32).
#pragma once

#include <cuda_bf16.h>

#include "jmix.h"
#include "poly_consts.cuh"

namespace jmix {

__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The normal distribution's Phi(v), and e = exp(-v^2 / 2) for its density.  Phi(-|v|) =
// t P(t) e, t = 1 / (1 + NC |v|), with the minimax polynomial P of poly_consts.cuh: 1.7e-7 of its
// value, and no difference from 1, so that small values keep their accuracy; e adds the
// roundings of v^2 / 2, up to 2^-16 at |v| = 12.  (A polynomial with an absolute bound, as
// Abramowitz and Stegun 7.1.26, is 0.4% off at -6 and 3% at -12, more than bf16's rounding; with
// three multiply-adds a value less, 4100 x 512 -> 4104 took 65 us, here 68, and 8192 x 4096 ->
// 14336 740 us, here 745, within its spread.)
__device__ __forceinline__ float normal_cdf(float v, float& e) {
  const float t = __fdividef(1.0f, fmaf(fabsf(v), poly::NC, 1.0f));
  float p = fmaf(t, poly::N7, poly::N6);
  p = fmaf(p, t, poly::N5);
  p = fmaf(p, t, poly::N4);
  p = fmaf(p, t, poly::N3);
  p = fmaf(p, t, poly::N2);
  p = fmaf(p, t, poly::N1);
  p = fmaf(p, t, poly::N0);
  e = __expf(-0.5f * v * v);
  const float tail = p * t * e;
  return v < 0.0f ? tail : 1.0f - tail;
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
