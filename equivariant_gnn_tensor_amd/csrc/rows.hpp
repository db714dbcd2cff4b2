// Building blocks of the row kernels: vector loads and stores of any alignment in
// fp32, bf16 and fp16, and sums over groups of lanes.
#pragma once

#include "common.hpp"
#include "wave.hpp"

namespace etpc {

template <class T, int N>
using VecN = T __attribute__((ext_vector_type(N)));
template <class T>
using Vec8 = VecN<T, 8>;

// Element types of the row operators (etpc_dtype).
using Bf16 = __bf16;
using F16 = _Float16;

// N = 4 or 8 elements of a row of n from column c on (a multiple of N), in two steps.
// fetch issues one vector load and waits for nothing: the last vector of a row that ends
// inside it is read as the row's last N elements.  settle, at the point of use, moves those
// down into place and clears what lies past the end (columns at and past n are 0).
// Element-wise loads of the row's end cost more than the whole rest of it (bf16 rows of
// 2047: 226 us against 63 for 2048, layer norm backward of 32768 rows).  The address only
// has to be aligned to the element: unaligned vector accesses are native here.  kEven: n is
// a multiple of N, so nothing ends inside a vector (and the code for it costs no registers).
template <int N, bool kEven, class T>
__device__ inline VecN<T, N> fetch(const T* __restrict__ p, int c, int n) {
  VecN<T, N> t = {};
  if (kEven) {
    if (c < n) __builtin_memcpy(&t, p + c, sizeof(t));
  } else if (n >= N) {
    if (c < n) __builtin_memcpy(&t, p + min(c, n - N), sizeof(t));
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (c + k < n) t[k] = p[c + k];
  }
  return t;
}

template <int N, bool kEven, class T>
__device__ inline void settle(const VecN<T, N>& t, int c, int n, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = static_cast<float>(t[k]);
  if (!kEven && n >= N && c + N > n && c < n) {
    const int down = c + N - n;   // 1 .. N - 1
#pragma unroll
    for (int by = 1; by < N; by *= 2)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = (down & by) ? (k + by < N ? v[k + by] : 0.f) : v[k];
  }
}

template <int N, bool kEven, class T>
__device__ inline void load(const T* __restrict__ p, int c, int n, float (&v)[N]) {
  settle<N, kEven, T>(fetch<N, kEven>(p, c, n), c, n, v);
}

// N elements of which `left` are the thread's own (zeros past them): for calls in place, where the elements
// before a row's last vector are being written by their own threads.
template <int N, class T>
__device__ inline void load_own(const T* p, int left, float (&v)[N]) {
  if (left >= N) {
    load<N, true>(p, 0, N, v);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = k < left ? static_cast<float>(p[k]) : 0.f;
  }
}

// Rounds to the element type here, once (to nearest, ties to even).  The end of a row goes
// out as at most three stores, of four, two and one elements.
template <int N, bool kEven, class T>
__device__ inline void store(T* __restrict__ p, int c, int n, const float (&v)[N]) {
  VecN<T, N> t;
#pragma unroll
  for (int k = 0; k < N; ++k) t[k] = static_cast<T>(v[k]);
  if (kEven ? c < n : c + N <= n) {
    __builtin_memcpy(p + c, &t, sizeof(t));
  } else if (!kEven && c < n) {
    const int left = n - c;   // 1 .. N - 1
    if (N == 8 && (left & 4)) {
      const VecN<T, 4> u = {t[0], t[1], t[2], t[3]};
      __builtin_memcpy(p + c, &u, sizeof(u));
    }
    if (left & 2) {
      const bool high = N == 8 && (left & 4);
      const VecN<T, 2> u = {high ? t[N - 4] : t[0], high ? t[N - 3] : t[1]};
      __builtin_memcpy(p + c + (left & 4), &u, sizeof(u));
    }
    if (left & 1) {
      const T low = (left & 2) ? t[2] : t[0], high = (left & 2) ? t[N - 2] : t[N - 4];
      p[n - 1] = N == 8 && (left & 4) ? high : low;
    }
  }
}

// The same for a result that is as large as the caches or larger and read by a later kernel: whole
// vectors go out past L2 (65408 x 4096 bf16 results of a product: 566 us with store, 542 with this,
// since what L2 keeps instead are the product's operands).
template <int N, class T>
__device__ inline void stream(T* __restrict__ p, int c, int n, const float (&v)[N]) {
  typedef T Piece __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  constexpr int E = 16 / sizeof(T);
  static_assert(N % E == 0, "whole 16-byte pieces");
  if (c + N <= n) {
#pragma unroll
    for (int i = 0; i < N; i += E) {
      Piece t;
#pragma unroll
      for (int k = 0; k < E; ++k) t[k] = static_cast<T>(v[i + k]);
      __builtin_nontemporal_store(t, reinterpret_cast<Piece*>(p + c + i));
    }
  } else {
    store<N, false>(p, c, n, v);
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

// Sums of N values over each group of G threads: lanes of one wave (G <= 64), or whole waves
// of the workgroup through `lds` ([2][kGroups][N][G / 64] floats, halves used in turn so
// one barrier a call is enough; every thread of the workgroup has to call).
template <int G, int kGroups, int N>
__device__ inline void group_sum(float (&v)[N], float* lds, int& half) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = lane_sum<(G < 64 ? G : 64)>(v[j]);
  if (G > 64) {
    constexpr int W = G / 64;
    float* buf = lds + (half * kGroups + (kGroups > 1 ? threadIdx.x / G : 0)) * N * W;
    half ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int j = 0; j < N; ++j) buf[j * W + (kGroups > 1 ? threadIdx.x / 64 % W : threadIdx.x / 64)] = v[j];
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

// 1 / sqrt(var + eps) from the sum of squares about a mean that is `off` too low.  A variance
// that rounding took below zero is zero; one that is NaN stays so (a maximum with zero would
// hide it), and with it every number of the row.
__device__ inline float norm_rstd(float squares, float off, float inv_n, float eps) {
  const float var = fmaf(squares, inv_n, -off * off);
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

// The mean to keep for the backward pass.  `off` corrects the rounding of a mean of the size
// of the spread and above.  Near zero it does not: all numbers of one binade round x - mean
// by the same amount, their average is that amount, and the sum it would correct is the
// better one (4096 normal numbers about 0: median relative error 1e-7 without, 6e-7 with;
// about 1/4 of their spread 3.1e-8 and 2.5e-8; about 300 spreads 3.0e-8 and 2.4e-8).  An
// infinite mean stays as it is: `off` is NaN then, and so is rstd.
__device__ inline float norm_mean(float mean, float off, float rstd) {
  return fabsf(mean) * rstd > 0.25f ? mean + off : mean;
}

// p[slice width] + p[(slice + kSlices) width] + ... over the first `parts` rows, in order, with
// eight loads in flight.
template <int kSlices>
__device__ inline float sum_slice(const float* __restrict__ p, int64_t width, int slice, int parts) {
  float s = 0.f;
  int q = slice;
  for (; q + 7 * kSlices < parts; q += 8 * kSlices) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[(q + i * kSlices) * width];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
#pragma unroll 4
  for (; q < parts; q += kSlices) s += p[q * width];
  return s;
}

}  // namespace etpc
