// Activations of the dense layer and their slopes, in fp32 (device code).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/etpc.h"

namespace etpc {

// exp(c x) and 1 / x to the accuracy the element type can hold.  16-bit results take the hardware's
// exp2 of the scaled argument (its product rounds to 2^-24 of itself) and reciprocal (one unit):
// far below their half step, and two instructions where the library's functions take twenty.
template <bool kWide>
__device__ inline float exp_of(float c, float x) {
  return kWide ? expf(c * x) : __builtin_amdgcn_exp2f(c * 1.44269504f * x);
}
template <bool kWide>
__device__ inline float inverse(float x) {
  return kWide ? 1.f / x : __builtin_amdgcn_rcpf(x);
}

// The logistic function; exp overflows to infinity on one side, which gives 0 as it should.
template <bool kWide>
__device__ inline float logistic(float x) {
  return inverse<kWide>(1.f + exp_of<kWide>(-1.f, x));
}

// For gelu: the tail Phi(-|z|) of the normal distribution, and e = exp(-z^2 / 2).  With a = |z| / sqrt 2
// the tail is erfc(a) / 2 = e f(a), and f is 1 / (1 + a / 2) times a polynomial in it, fitted by
// least squares reweighted towards the smallest relative error (1e-7 over 0 <= a <= 16 with these
// coefficients, 4e-7 with its evaluation in fp32).  It does not cancel like 1 + erf, and takes a third of
// the library's erfc.  fp32 rows, bound by their products, take erfc.
template <bool kWide>
__device__ inline float normal_tail(float z, float& e) {
  e = exp_of<kWide>(-0.5f, z * z);
  if (kWide) return 0.5f * erfcf(0.70710678f * fabsf(z));
  const float t = inverse<kWide>(fmaf(0.35355339f, fabsf(z), 1.f));
  float p = -0.029572323f;
  p = fmaf(p, t, 0.142542049f);
  p = fmaf(p, t, -0.244266406f);
  p = fmaf(p, t, 0.139947891f);
  p = fmaf(p, t, -0.0140409898f);
  p = fmaf(p, t, 0.10168989f);
  p = fmaf(p, t, 0.121455595f);
  p = fmaf(p, t, 0.141201928f);
  p = fmaf(p, t, 0.141042352f);
  return p * t * e;
}

// tanh by one exp; near zero, where 1 - 2 / (..) cancels, its series.
template <bool kWide>
__device__ inline float act_tanh(float z) {
  if (kWide) return tanhf(z);
  const float s = z * z, r = fmaf(-2.f, inverse<kWide>(1.f + exp_of<kWide>(2.f, z)), 1.f);
  return s < 0.09f ? z * fmaf(s, fmaf(s, fmaf(s, fmaf(s, 0.021869489f, -0.053968254f), 0.13333333f), -0.33333333f), 1.f) : r;
}

// A factor that would be infinite beside a zero is bounded (fminf, fmaxf): silu and gelu of -inf are
// 0 and their slopes at +-inf 1 and 0.  Those drop a NaN, but the other factor keeps it.
template <bool kWide, int N>
__device__ inline void activate(float (&v)[N], int act) {
  if (act == ETPC_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = v[k] < 0.f ? 0.f : v[k];
  } else if (act == ETPC_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = fmaxf(v[k], -200.f) * logistic<kWide>(v[k]);
  } else if (act == ETPC_ACT_GELU) {   // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float e;
      const float tail = normal_tail<kWide>(v[k], e);
      v[k] = fmaf(-fminf(fabsf(v[k]), 200.f), tail, fmaxf(v[k], 0.f));
    }
  } else if (act == ETPC_ACT_TANH) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = act_tanh<kWide>(v[k]);
  }
}

// v times the slope at z.
template <bool kWide, int N>
__device__ inline void times_slope(float (&v)[N], const float (&z)[N], int act) {
  if (act == ETPC_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] *= z[k] <= 0.f ? 0.f : z[k] == z[k] ? 1.f : z[k];
  } else if (act == ETPC_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float p = logistic<kWide>(z[k]);
      v[k] *= p * fmaf(fminf(fmaxf(z[k], -200.f), 200.f), 1.f - p, 1.f);
    }
  } else if (act == ETPC_ACT_GELU) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float e;
      const float tail = normal_tail<kWide>(z[k], e);
      v[k] *= fmaf(fminf(fmaxf(z[k], -200.f), 200.f) * 0.39894228f, e, z[k] > 0.f ? 1.f - tail : tail);
    }
  } else if (act == ETPC_ACT_TANH) {
    // 1 - tanh^2 = 4 e / (1 + e)^2 with e = exp(-2 |z|); the difference would leave nothing of a slope below 2^-24
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float e = exp_of<kWide>(-2.f, fabsf(z[k])), r = inverse<kWide>(1.f + e);
      v[k] *= 4.f * e * r * r;
    }
  }
}

}  // namespace etpc
