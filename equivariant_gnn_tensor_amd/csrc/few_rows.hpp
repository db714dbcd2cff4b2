// The dense layer for one or two rows (templates; few_rows.hip holds the launches).
//
//   C(m, n) = epilogue(sum_k A(m, k) B(k, n)),  m < 2
//
// The weights are read once and nothing else counts, so this is about having enough of them on
// their way at once: no matrix instructions, no slices, one pass with up to eight 16-byte loads a lane in
// flight.  The rows wait in LDS as fp32, 2048 k at a time.
//   along:  weights contiguous in k.  A wave owns kOwn outputs, its lanes take 16-byte pieces of k, the
//           sums are added over the wave at the end.
//   across: weights contiguous in n.  Eight lanes take 128 bytes of n of one k (four take 64), a wave eight
//           (sixteen) k and a workgroup 128 (256); the sums are added over lanes, then over waves in LDS.
// fp32 sums in a fixed order.  From three rows on the tiles of matmul.hpp are faster (eight rows of 4096 ->
// 4096 bf16: 56 and 74 us here, along and across, where conversions and multiply-adds count; 14 there).  1 x 1024 -> 1024
// fp32 (4 MB of weights, across): 5.5 us with the weights from memory.
#pragma once

#include "activation.hpp"
#include "linear.hpp"
#include "rows.hpp"

namespace etpc {
namespace few {

constexpr int kBlock = 2048;   // k of a pass over LDS

// The rows' k from k0 on as fp32, zeros past K.
template <class T, int M>
__device__ inline void stage(float (*lds)[kBlock], const MatmulArgs& a, int k0) {
  const int n = min(kBlock, a.K - k0), padded = (n + 127) / 128 * 128;
  for (int m = 0; m < M; ++m)
    for (int k = threadIdx.x; k < padded; k += blockDim.x)
      lds[m][k] = m < a.M && k < n ? static_cast<float>(static_cast<const T*>(a.a)[m * a.lda + k0 + k]) : 0.f;
}

template <class T>
__device__ inline void finish(const MatmulArgs& a, int m, int n, float v) {
  if (a.bias != nullptr) v += a.bias[n];
  if (a.z != nullptr) static_cast<T*>(a.z)[m * a.ldz + n] = static_cast<T>(v);
  float y[1] = {v};
  if (a.act != ETPC_ACT_NONE) activate<sizeof(T) == 4>(y, a.act);
  if (a.res != nullptr) y[0] += static_cast<float>(static_cast<const T*>(a.res)[m * a.ldres + n]);
  static_cast<T*>(a.c)[m * a.ldc + n] = static_cast<T>(y[0]);
}

constexpr int kAlongThreads = 256;
template <class T, int M, int kOwn>
__global__ __launch_bounds__(kAlongThreads) void along_kernel(const MatmulArgs a) {
  constexpr int E = 16 / sizeof(T);
  __shared__ float rows[M][kBlock];
  const int lane = threadIdx.x & 63;
  constexpr int kGroup = kAlongThreads / 64 * kOwn;   // outputs of a workgroup, which walks on past a launch's most
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGroup; first < a.N; first += static_cast<int64_t>(gridDim.x) * kGroup) {
    const int64_t n0 = first + (threadIdx.x >> 6) * kOwn;
    float sum[kOwn][M] = {};
    for (int k0 = 0; k0 < a.K; k0 += kBlock) {
      __syncthreads();
      stage<T, M>(rows, a, k0);
      __syncthreads();
      const int n = min(kBlock, a.K - k0);
#pragma unroll 2
      for (int k = lane * E; k < n; k += 64 * E) {
        float w[kOwn][E];
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
          const int64_t row = min(n0 + o, static_cast<int64_t>(a.N) - 1);
          load<E, false>(static_cast<const T*>(a.b) + row * a.ldb, k0 + k, a.K, w[o]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float x = rows[m][k + e];
#pragma unroll
            for (int o = 0; o < kOwn; ++o) sum[o][m] = fmaf(x, w[o][e], sum[o][m]);
          }
      }
    }
#pragma unroll
    for (int o = 0; o < kOwn; ++o)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float v = lane_sum<64>(sum[o][m]);
        if (lane == o * M + m && m < a.M && n0 + o < a.N) finish<T>(a, m, static_cast<int>(n0) + o, v);
      }
  }
}

constexpr int kAcrossThreads = 1024;
template <class T, int M, int kLanes>
__global__ __launch_bounds__(kAcrossThreads) void across_kernel(const MatmulArgs a) {
  constexpr int E = 16 / sizeof(T), kCols = kLanes * E, kWaves = kAcrossThreads / 64, kDeep = 64 / kLanes;
  static_assert(kLanes == 8 || kLanes == 4, "the sums over lanes below");
  constexpr int kStaged = M * kBlock, kSums = kWaves * M * kCols;
  __shared__ float lds[kStaged > kSums ? kStaged : kSums];
  float(*const rows)[kBlock] = reinterpret_cast<float(*)[kBlock]>(lds);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int mine = wave * kDeep + lane / kLanes;
  for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCols; n0 < a.N; n0 += static_cast<int64_t>(gridDim.x) * kCols) {
    const int n = static_cast<int>(n0) + lane % kLanes * E;
    float sum[M][E] = {};
    for (int k0 = 0; k0 < a.K; k0 += kBlock) {
      __syncthreads();
      stage<T, M>(rows, a, k0);
      __syncthreads();
      const int count = min(kBlock, a.K - k0);
#pragma unroll 8
      for (int k = mine; k < count; k += kWaves * kDeep) {
        float w[E];
        load<E, false>(static_cast<const T*>(a.b) + (k0 + k) * a.ldb, n, a.N, w);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float x = rows[m][k];
#pragma unroll
          for (int e = 0; e < E; ++e) sum[m][e] = fmaf(x, w[e], sum[m][e]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // over the k of the wave: lanes kLanes, 2 kLanes, ... and 32 apart
        float v = sum[m][e];
        v += dpp_f<0x128>(v);   // rotation by eight in each row of sixteen
        if (kLanes == 4) v += dpp_f<0x124>(v);
        v = add_lane16(v);
        v = add_lane32(v);
        if (lane < kLanes) lds[(wave * M + m) * kCols + lane * E + e] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < M * kCols; i += kAcrossThreads) {
      const int m = i / kCols, c = i % kCols;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) v += lds[(q * M + m) * kCols + c];
      if (m < a.M && n0 + c < a.N) finish<T>(a, m, static_cast<int>(n0) + c, v);
    }
  }
}

}  // namespace few
}  // namespace etpc
