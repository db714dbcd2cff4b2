// Activations of the dense layer and their slopes, in fp32 (device code).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/etpc.h"

namespace etpc {

// exp to the accuracy the element type can hold: 16-bit results take the hardware's exp2 of
// the scaled argument (its product rounds to 2^-24 |x|, far below their half step).
template <bool kWide>
__device__ inline float act_exp(float x) {
  return kWide ? expf(x) : __expf(x);
}

// The logistic function; exp overflows to infinity on one side, which gives 0 as it should.
template <bool kWide>
__device__ inline float logistic(float x) {
  const float e = 1.f + act_exp<kWide>(-x);
  return kWide ? 1.f / e : __frcp_rn(e);
}

// Both limits are taken where the formulas would multiply zero by infinity: silu and gelu of
// -inf are -0 and their slopes at +-inf 1 and 0.  NaN passes through every comparison.
template <bool kWide, int N>
__device__ inline void activate(float (&v)[N], int act) {
  if (act == ETPC_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = v[k] < 0.f ? 0.f : v[k];
  } else if (act == ETPC_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = v[k] < -200.f ? -0.f : v[k] * logistic<kWide>(v[k]);
  } else if (act == ETPC_ACT_GELU) {   // z Phi(z), by erfc: 1 + erf would cancel below zero
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = v[k] < -200.f ? -0.f : 0.5f * v[k] * erfcf(-0.70710678f * v[k]);
  } else if (act == ETPC_ACT_TANH) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = tanhf(v[k]);
  }
}

template <bool kWide>
__device__ inline float slope(float z, int act) {
  switch (act) {
    case ETPC_ACT_RELU:
      return z <= 0.f ? 0.f : z == z ? 1.f : z;
    case ETPC_ACT_SILU: {
      const float c = z > 200.f ? 200.f : z < -200.f ? -200.f : z;
      const float p = logistic<kWide>(c);
      return p * (1.f + c * (1.f - p));
    }
    case ETPC_ACT_GELU: {
      const float c = z > 200.f ? 200.f : z < -200.f ? -200.f : z;
      return 0.5f * erfcf(-0.70710678f * c) + c * 0.39894228f * act_exp<kWide>(-0.5f * c * c);
    }
    case ETPC_ACT_TANH: {
      const float t = tanhf(z);
      return 1.f - t * t;
    }
    default:
      return 1.f;
  }
}

}  // namespace etpc
