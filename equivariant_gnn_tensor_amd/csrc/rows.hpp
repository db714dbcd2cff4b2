// Building blocks of the row kernels: eight-element loads and stores of any alignment in
// fp32, bf16 and fp16, and sums over groups of lanes.
#pragma once

#include "common.hpp"
#include "wave.hpp"

namespace etpc {

template <class T>
using Vec8 = T __attribute__((ext_vector_type(8)));
using Float8 = Vec8<float>;

// Element types of the row operators (etpc_dtype).
using Bf16 = __bf16;
using F16 = _Float16;

// Eight elements of a row from column c on; columns at and past n read as 0.  The address
// only has to be aligned to the element: unaligned vector accesses are native here, so
// odd row lengths and strides run the same code as even ones.
template <class T>
__device__ inline void load8(const T* __restrict__ p, int c, int n, float (&v)[8]) {
  if (c + 8 <= n) {
    Vec8<T> t;
    __builtin_memcpy(&t, p + c, sizeof(t));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(t[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c + k < n ? static_cast<float>(p[c + k]) : 0.f;
  }
}

// Rounds to the element type here, once (to nearest, ties to even).
template <class T>
__device__ inline void store8(T* __restrict__ p, int c, int n, const float (&v)[8]) {
  if (c + 8 <= n) {
    Vec8<T> t;
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = static_cast<T>(v[k]);
    __builtin_memcpy(p + c, &t, sizeof(t));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < n) p[c + k] = static_cast<T>(v[k]);
  }
}

// v + its value in the lane 16 (32) away: the swap instructions exchange 16-lane rows
// (wave halves) between two registers, so the sum of both results is the pair's sum.
__device__ inline float add_lane16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  return __int_as_float(r[0]) + __int_as_float(r[1]);
}
__device__ inline float add_lane32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return __int_as_float(r[0]) + __int_as_float(r[1]);
}

// Sum over aligned groups of G lanes (a power of two up to 64); every lane gets it, with
// the same bits.  Whole groups have to be active.
template <int G>
__device__ inline float lane_sum(float v) {
  if (G >= 2) v += dpp_f<0xB1>(v);    // lane ^ 1
  if (G >= 4) v += dpp_f<0x4E>(v);    // lane ^ 2
  if (G >= 8) v += dpp_f<0x141>(v);   // the other four of eight
  if (G >= 16) v += dpp_f<0x140>(v);  // the other eight of sixteen
  if (G >= 32) v = add_lane16(v);
  if (G >= 64) v = add_lane32(v);
  return v;
}

// Sums of N values over a group of G threads: lanes of one wave (G <= 64), or the whole
// workgroup of G threads through `lds` ([2][N][G / 64] floats, halves used in turn so one
// barrier a call is enough).
template <int G, int N>
__device__ inline void group_sum(float (&v)[N], float* lds, int& half) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = lane_sum<(G < 64 ? G : 64)>(v[j]);
  if (G > 64) {
    constexpr int W = G / 64;
    float* buf = lds + half * N * W;
    half ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int j = 0; j < N; ++j) buf[j * W + threadIdx.x / 64] = v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) s += buf[j * W + i];
      v[j] = s;
    }
  }
}

}  // namespace etpc
