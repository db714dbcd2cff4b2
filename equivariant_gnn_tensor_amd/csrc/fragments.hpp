// Fragments of the matrix instructions: 16-byte chunks of rows and their products (device code).
#pragma once

#include "rows.hpp"

namespace etpc {
namespace mm {

typedef float Acc __attribute__((ext_vector_type(16)));
typedef uint32_t Chunk __attribute__((ext_vector_type(4)));   // 16 bytes
typedef short Tr4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void LdsVoid;
typedef __attribute__((address_space(3))) Tr4 LdsTr4;

constexpr int kSliceBytes = 128;
template <class T>
constexpr int slice() {
  return kSliceBytes / static_cast<int>(sizeof(T));
}

// Elements c .. of a row of n as 16 bytes; zero past the end.
template <class T>
__device__ inline Chunk fetch_chunk(const T* __restrict__ row, int c, int n) {
  constexpr int E = 16 / sizeof(T);
  Chunk t = {};
  if (c >= n) return t;
  if (n >= E) {
    const int at = min(c, n - E);
    __builtin_memcpy(&t, row + at, 16);
    if (at != c) {
      unsigned __int128 v;
      __builtin_memcpy(&v, &t, 16);
      v >>= (c - at) * 8 * static_cast<int>(sizeof(T));
      __builtin_memcpy(&t, &v, 16);
    }
  } else {
    T e[E] = {};
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < n) e[k] = row[c + k];
    __builtin_memcpy(&t, e, 16);
  }
  return t;
}

// acc + the products of two fragments, eight k (16 bits) or four (fp32) a lane and wave half.
template <class T>
__device__ inline Acc multiply(const Chunk& b, const Chunk& a, Acc acc) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(b[j]), __uint_as_float(a[j]), acc, 0, 0, 0);
    return acc;
  } else {
    Vec8<T> x, y;
    __builtin_memcpy(&x, &b, 16);
    __builtin_memcpy(&y, &a, 16);
    if constexpr (__is_same(T, F16))
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, acc, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, acc, 0, 0, 0);
  }
}

}  // namespace mm
}  // namespace etpc
