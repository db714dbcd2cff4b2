// The dense layer between narrow rows (up to 128 numbers, see fits_fwd and fits_bwd), forward and backward (templates; narrow_*.hip
// hold the instantiations of one element type each).
//
//   forward:  z = x w + b, y = act(z) + residual
//   backward: z_bar = y_bar act'(z), x_bar = z_bar w^T, w_bar = x^T z_bar, b_bar = column sums of z_bar
//
// Memory bound (214980 rows of 64: 20 flop a byte), so every row is read once, the weights stay in
// LDS, and a wave works through 32 rows at a time on its own, without a barrier: lane r (and r + 32)
// loads row r's 16-byte chunks straight into the fragments of the matrix instructions, the next
// rows' while these are worked on.  With the weights' fragment first, a lane gets four adjacent
// columns of one row; swapping wave halves makes that eight, which are loaded and stored as one.
//
// The backward pass is one kernel: z_bar and x go through a few KB of LDS of the wave.  x_bar's fragments of
// z_bar are read back as they were written, w_bar's, whose contraction runs over rows, transposed.  The
// matrix cores take 16-bit numbers of z_bar, so it goes into both products as the sum of two of them, the
// rounded one and what that leaves (off by 2^-16 of z_bar in bf16, 2^-22 in fp16): one rounding alone takes the
// gradients from 0.0017 to 0.0023 off (root mean square, bf16; their own rounding is 0.0017) and saves 2 of 44
// us.  w_bar's and b_bar's sums stay in registers over all of a wave's rows, are added up
// over the workgroup's waves in LDS and leave one partial sum a workgroup, added in a fixed order
// by a second launch.
//
// 214980 x 64 -> 64 bf16 silu: forward 21 us a call (82.6 MB, 3.9 TB/s; half of a wave's cycles are
// waits), backward 44 (110 MB; 41.5 and the second launch's 4.7), bound by conversions, slopes and the way
// through LDS.  16-bit rows that are not whole chunks spill 25 registers backward with 64 -> 64, 21 with 128 -> 32
// and a slope, 5 without (63 -> 63 silu 80 us).
#pragma once

#include <algorithm>

#include "activation.hpp"
#include "fragments.hpp"
#include "narrow_args.hpp"
#include "rows.hpp"

namespace etpc {
namespace narrow {

using mm::Acc;
using mm::Chunk;

// Chunks of 32-byte steps: a step holds two chunks of a row, one for each half of the wave.
template <class T>
constexpr int steps(int tiles) {
  return tiles * static_cast<int>(sizeof(T));
}
// LDS of weights as rows of 128-byte slices, chunk c of row r at c ^ (r / 2 mod 8) (see matmul.hpp).
template <class T>
constexpr int slices(int tiles) {
  return (steps<T>(tiles) + 3) / 4;
}
__device__ inline int weight_at(int rows, int r, int chunk) {
  return (chunk >> 3) * rows * 128 + r * 128 + (((chunk & 7) ^ ((r >> 1) & 7)) << 4);
}

// Row r, numbers k .. of the weights: w[r ld + k] (`along`) or w[k ld + r]; zero past n rows, K numbers.
template <class T>
__device__ inline void fill_weights(char* lds, int rows, int chunks, const T* __restrict__ w, int64_t ld, bool along,
                                    int n, int K) {
  constexpr int E = 16 / sizeof(T);
  for (int q = threadIdx.x; q < rows * chunks; q += blockDim.x) {
    const int r = q % rows, c = q / rows;
    Chunk t = {};
    if (r < n) {
      if (along) {
        t = mm::fetch_chunk(w + r * ld, c * E, K);
      } else {
        T e[E] = {};
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (c * E + k < K) e[k] = w[(c * E + k) * ld + r];
        __builtin_memcpy(&t, e, 16);
      }
    }
    *reinterpret_cast<Chunk*>(lds + weight_at(rows, r, c)) = t;
  }
}

// The chunks of a row that a lane holds: chunk 2 s + h of row r for each step s.
template <class T, int S, bool kEven>
struct RowChunks {
  Chunk c[S];
  __device__ inline void read(const void* p, int64_t at, int n, int h) {
    constexpr int E = 16 / sizeof(T);
    const T* row = static_cast<const T*>(p) + at;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = (2 * s + h) * E;
      if (kEven) {
        c[s] = Chunk{};
        if (k < n) __builtin_memcpy(&c[s], row + k, 16);
      } else {
        c[s] = mm::fetch_chunk(row, k, n);
      }
    }
  }
};

// Eight adjacent columns of a lane's row from the results of one 32-column tile: g = 0, 1 are columns
// 16 g + 8 h ...  Halves of the wave hold four columns each; lanes 0 to 31 keep the first eight of
// sixteen, lanes 32 to 63 the others.
__device__ inline void eight(const Acc& acc, int g, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_int(acc[8 * g + k]), __float_as_int(acc[8 * g + 4 + k]), false, false);
    v[k] = __int_as_float(r[0]);
    v[4 + k] = __int_as_float(r[1]);
  }
}

// A wave's 32 result rows, TILES 32-column tiles wide, on their way out: a lane holds four columns of one row
// at a time, and they are turned over in LDS (fp32, chunks of four) to eight columns a lane and whole row
// segments a pass, where the rest is plain row code (214980 x 64 -> 64 bf16 silu 21.1 us; 24.7 storing 32
// bytes of a row at a time from `eight`, with the activations' code in every column's place).
template <int TILES>
struct RowsOut {
  static constexpr int C = TILES * 8, kVecs = TILES * 4;   // chunks of a row; eights of a row
  static constexpr int kBytes = 32 * C * 16;
  static __device__ inline int at(int r, int c) { return (r * C + (c ^ (C == 8 ? (r >> 1) & 7 : r & 15))) << 4; }
  static __device__ inline void put(char* lds, int tile, const Acc& acc, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const VecN<float, 4> v = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
      *reinterpret_cast<VecN<float, 4>*>(lds + at(lane & 31, 8 * tile + 2 * q + (lane >> 5))) = v;
    }
  }
  // f(row, column, eight numbers) for each of a lane's vectors
  template <class F>
  static __device__ inline void each(const char* lds, int lane, F&& f) {
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int p = 0; p < kVecs / 2; ++p) {
      const int q = p * 64 + lane, r = q / kVecs, c = q % kVecs * 2;
      float v[8];
      __builtin_memcpy(v, lds + at(r, c), 16);
      __builtin_memcpy(v + 4, lds + at(r, c + 1), 16);
      f(r, 4 * c, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
};

constexpr int kFwdThreads = 256;

template <class T, int IT, int OT, bool kEven>
__global__ __launch_bounds__(kFwdThreads) void fwd_kernel(const FwdArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int S = steps<T>(IT), kRows = 32 * OT;
  __shared__ __attribute__((aligned(16))) char w[slices<T>(IT) * kRows * 128];
  using Out = RowsOut<OT>;
  __shared__ __attribute__((aligned(16))) char out[Out::kBytes * kFwdThreads / 64];
  char* const turn = out + (threadIdx.x >> 6) * Out::kBytes;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int64_t tiles = (static_cast<int64_t>(a.rows) + 31) / 32, step = static_cast<int64_t>(gridDim.x) * (kFwdThreads / 64);
  int64_t tile = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / 64) + (threadIdx.x >> 6);
  const auto row_of = [&](int64_t t) __attribute__((always_inline)) {
    return min(t * 32 + (lane & 31), static_cast<int64_t>(a.rows) - 1);
  };
  RowChunks<T, S, kEven> next;
  if (tile < tiles) next.read(a.x, row_of(tile) * a.xs, a.n_in, h);
  fill_weights(w, kRows, 2 * S, static_cast<const T*>(a.w), a.ldw, !a.by_out, a.n_out, a.n_in);
  __syncthreads();
  for (; tile < tiles; tile += step) {
    const RowChunks<T, S, kEven> now = next;
    if (tile + step < tiles) next.read(a.x, row_of(tile + step) * a.xs, a.n_in, h);
    if (IT * OT * sizeof(T) > 8) asm volatile("" ::: "memory");   // the weights stay in LDS: registers do not hold them
    Acc acc[OT] = {};
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int j = 0; j < OT; ++j) {
        const Chunk f = *reinterpret_cast<const Chunk*>(w + weight_at(kRows, 32 * j + (lane & 31), 2 * s + h));
        acc[j] = mm::multiply<T>(f, now.c[s], acc[j]);
      }
#pragma unroll
    for (int j = 0; j < OT; ++j) Out::put(turn, j, acc[j], lane);
    Out::each(turn, lane, [&](int r, int n, float (&v)[8]) __attribute__((always_inline)) {
      const int64_t m = tile * 32 + r;
      if (m >= a.rows || n >= a.n_out) return;
      float b[8];
      if (a.b != nullptr) {
        load<8, false>(a.b, n, a.n_out, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
      }
      if (a.z != nullptr) store<8, false>(static_cast<T*>(a.z) + m * a.zs, n, a.n_out, v);
      if (a.act != ETPC_ACT_NONE) activate<sizeof(T) == 4>(v, a.act);
      if (a.res != nullptr) {
        load<8, false>(static_cast<const T*>(a.res) + m * a.ress, n, a.n_out, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
      }
      store<8, false>(static_cast<T*>(a.y) + m * a.ys, n, a.n_out, v);
    });
  }
#endif
}

// ---------------------------------------------------------------- backward
// A wave's 32 rows of C chunks on their way through LDS.  Written a chunk of 16 rows at a time; read
// transposed, four rows of two 32-byte blocks (16 bits) or two rows of 32 numbers (fp32): the
// exclusive or spreads the first over half the banks, the others over all (fp32 rows of 32: half).
template <class T, int C>
__device__ inline int tile_at(int r, int c) {
  const int f = sizeof(T) == 2 ? (C == 8 ? (r & 2) << 1 | (r & 4) >> 1 : (r & 3) << 2 | (r & 4) >> 1)
                : C == 8       ? (r >> 1) & 7
                               : (r & 3) | (r & 4) << 1 | (r & 8) >> 1;
  return r * (C * 16) + ((c ^ f) << 4);
}
// Fragment of columns at .. at + 31 with rows as k (rows 16 s .. for 16 bits, 8 s .. for fp32).
template <class T, int C>
__device__ inline Chunk column_fragment(const char* lds, int at, int s, int lane) {
  Chunk t;
  if constexpr (sizeof(T) == 2) {
    const int k = 16 * s + 8 * (lane >> 5) + ((lane & 15) >> 2), col = at + (lane & 16) + (lane & 3) * 4;
    const mm::Tr4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm::LdsTr4*)(lds + tile_at<T, C>(k, col >> 3) + (col & 7) * 2));
    const mm::Tr4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm::LdsTr4*)(lds + tile_at<T, C>(k + 4, col >> 3) + (col & 7) * 2));
    __builtin_memcpy(&t, &lo, 8);
    __builtin_memcpy(reinterpret_cast<char*>(&t) + 8, &hi, 8);
  } else {
    const int col = at + (lane & 31);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      t[j] = *reinterpret_cast<const uint32_t*>(lds + tile_at<T, C>(8 * s + 4 * (lane >> 5) + j, col >> 2) + (col & 3) * 4);
  }
  return t;
}

// Eight waves, two a SIMD with 256 registers each; fp32 rows fill LDS with four.
template <class T>
constexpr int bwd_threads() {
  return sizeof(T) == 4 ? 256 : 512;
}

// kSlope: there is an activation, so z_bar is not y_bar.
template <class T, int IT, int OT, bool kEven, bool kSlope>
__global__ __launch_bounds__(bwd_threads<T>()) void bwd_kernel(const BwdArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int SI = steps<T>(IT), SO = steps<T>(OT), kWaves = bwd_threads<T>() / 64, E = 16 / sizeof(T);
  constexpr int kRows = 32 * IT;
  constexpr int CI = 2 * SI < 8 ? 8 : 2 * SI, CO = 2 * SO < 8 ? 8 : 2 * SO;   // chunks of a row in LDS
  constexpr int kParts = sizeof(T) == 2 && kSlope ? 2 : 1;   // numbers that z_bar is the sum of
  constexpr int kWeights = slices<T>(OT) * kRows * 128, kTile = 32 * 16 * (CI + kParts * CO);
  constexpr int kSums = IT * OT * 32 * 32 + OT * 32;   // numbers of a partial sum (padded)
  constexpr int kTiles = kTile * kWaves, kHalf = kSums * 4 * (kWaves / 2);
  __shared__ __attribute__((aligned(16))) char w[kWeights];
  __shared__ __attribute__((aligned(16))) char space[kTiles > kHalf ? kTiles : kHalf];
  const int lane = threadIdx.x & 63, h = lane >> 5, wave = threadIdx.x >> 6;
  char* const xt = space + wave * kTile;
  char* const zt = xt + 32 * 16 * CI;
  const int64_t tiles = (static_cast<int64_t>(a.rows) + 31) / 32, step = static_cast<int64_t>(gridDim.x) * kWaves;
  int64_t tile = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  const bool sums = a.part != nullptr, w_sums = a.w_sums;
  struct Rows {
    RowChunks<T, SI, kEven> x;
    RowChunks<T, SO, kEven> y_bar, z;
  } next;
  const auto read = [&](int64_t t) __attribute__((always_inline)) {
    const int64_t r = min(t * 32 + (lane & 31), static_cast<int64_t>(a.rows) - 1);
    next.y_bar.read(a.y_bar, r * a.ybs, a.n_out, h);
    if (kSlope) next.z.read(a.z, r * a.zs, a.n_out, h);
    if (w_sums) next.x.read(a.x, r * a.xs, a.n_in, h);
  };
  if (tile < tiles) read(tile);
  if (a.x_bar != nullptr)
    fill_weights(w, kRows, 2 * SO, static_cast<const T*>(a.w), a.ldw, a.by_out, a.n_in, a.n_out);
  __syncthreads();
  Acc wb[IT][OT] = {};
  float bb[SO][E] = {};   // sums over this lane's rows of its chunks
  const int first_lane = lane;
  for (; tile < tiles; tile += step) {
    // Four tiles of w_bar leave no registers for addresses in LDS, which would be kept and spilled: they are
    // computed again for each 32 rows (214980 x 64 -> 64 bf16 silu 40 us; 47 with 12 registers spilled).
    int lane = first_lane;
    if (sizeof(T) == 2 && IT * OT > 2) asm volatile("" : "+v"(lane));
    const int h = lane >> 5;
    const Rows now = next;
    if (sizeof(T) == 4 && tile + step < tiles) read(tile + step);
    // A row past the end is the last one again: cleared, as it may hold infinities, and counted as zero.
    const bool row = tile * 32 + (lane & 31) < a.rows;
    if (w_sums) {
#pragma unroll
      for (int s = 0; s < SI; ++s) *reinterpret_cast<Chunk*>(xt + tile_at<T, CI>(lane & 31, 2 * s + h)) = row ? now.x.c[s] : Chunk{};
    }
#pragma unroll
    for (int s = 0; s < SO; ++s) {
      const Chunk y = row ? now.y_bar.c[s] : Chunk{};
      T e[E];
      float v[E];
      __builtin_memcpy(e, &y, 16);
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = static_cast<float>(e[k]);
      if (kSlope) {
        const Chunk c = row ? now.z.c[s] : Chunk{};
        T ez[E];
        float z[E];
        __builtin_memcpy(ez, &c, 16);
#pragma unroll
        for (int k = 0; k < E; ++k) z[k] = static_cast<float>(ez[k]);
        times_slope<sizeof(T) == 4>(v, z, a.act);
      }
#pragma unroll
      for (int k = 0; k < E; ++k) bb[s][k] += v[k];
      if constexpr (kParts == 2) {
        // The first part is kept finite: the rest alone holds an infinity or a NaN, and what fp16 overflows by.
        constexpr float kTop = __is_same(T, F16) ? 65504.f : 3.3895314e38f;
        T rest[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
          e[k] = static_cast<T>(__builtin_amdgcn_fmed3f(v[k], -kTop, kTop));
          rest[k] = static_cast<T>(v[k] - static_cast<float>(e[k]));
        }
        Chunk t;
        __builtin_memcpy(&t, rest, 16);
        *reinterpret_cast<Chunk*>(zt + 32 * 16 * CO + tile_at<T, CO>(lane & 31, 2 * s + h)) = t;
      } else if (kSlope) {
#pragma unroll
        for (int k = 0; k < E; ++k) e[k] = static_cast<T>(v[k]);
      }
      Chunk t;
      __builtin_memcpy(&t, e, 16);
      *reinterpret_cast<Chunk*>(zt + tile_at<T, CO>(lane & 31, 2 * s + h)) = t;
    }
    __builtin_amdgcn_sched_barrier(0);
    if (sizeof(T) == 2 && tile + step < tiles) read(tile + step);   // there were no registers for it before
    asm volatile("" ::: "memory");   // the weights stay in LDS
    if (a.x_bar != nullptr) {
      const int64_t m = tile * 32 + (lane & 31);
      Acc acc[IT] = {};
#pragma unroll
      for (int s = 0; s < SO; ++s) {
        Chunk z[kParts];
#pragma unroll
        for (int p = 0; p < kParts; ++p) z[p] = *reinterpret_cast<const Chunk*>(zt + p * 32 * 16 * CO + tile_at<T, CO>(lane & 31, 2 * s + h));
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const Chunk f = *reinterpret_cast<const Chunk*>(w + weight_at(kRows, 32 * i + (lane & 31), 2 * s + h));
#pragma unroll
          for (int p = 0; p < kParts; ++p) acc[i] = mm::multiply<T>(f, z[p], acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int g = 0; g < 2; ++g) {   // stored as they are: turned over like the forward pass 45.6 us for 38.3, before z_bar had its rest
          const int n = 32 * i + 16 * g + 8 * h;
          float v[8];
          eight(acc[i], g, v);
          if (row && n < a.n_in) store<8, false>(static_cast<T*>(a.x_bar) + m * a.xbs, n, a.n_in, v);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (w_sums) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int s = 0; s < static_cast<int>(sizeof(T)); ++s) {
        Chunk fx[IT], fz[OT];
#pragma unroll
        for (int i = 0; i < IT; ++i) fx[i] = column_fragment<T, CI>(xt, 32 * i, s, lane);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
#pragma unroll
          for (int o = 0; o < OT; ++o) fz[o] = column_fragment<T, CO>(zt + p * 32 * 16 * CO, 32 * o, s, lane);
#pragma unroll
          for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int o = 0; o < OT; ++o) wb[i][o] = mm::multiply<T>(fz[o], fx[i], wb[i][o]);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  if (!sums) return;

  // ---- the workgroup's sums: the upper half of the waves hands its own to the lower half, and again
  const auto each = [&](float* at, bool add) __attribute__((always_inline)) {   // registers to LDS, or LDS added to them
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int o = 0; o < OT; ++o)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float* p = at + ((i * OT + o) * 4 + q) * 256 + 4 * lane;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (add) wb[i][o][4 * q + k] += p[k];
            else p[k] = wb[i][o][4 * q + k];
          }
        }
    float* p = at + IT * OT * 1024;
    if ((lane & 31) == 0)
#pragma unroll
      for (int s = 0; s < SO; ++s)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          if (add) bb[s][k] += p[(2 * s + h) * E + k];
          else p[(2 * s + h) * E + k] = bb[s][k];
        }
  };
#pragma unroll
  for (int s = 0; s < SO; ++s)
#pragma unroll
    for (int k = 0; k < E; ++k) bb[s][k] = lane_sum<32>(bb[s][k]);
#pragma unroll
  for (int by = kWaves / 2; by > 0; by /= 2) {
    __syncthreads();
    float* const at = reinterpret_cast<float*>(space);
    if (wave >= by && wave < 2 * by) each(at + (wave - by) * kSums, false);
    __syncthreads();
    if (wave < by) each(at + wave * kSums, true);
  }
  if (wave != 0) return;
  // part[workgroup]: [n_in][n_out] (or [n_out][n_in] with !wb_by_out), then [n_out]
  float* const out = a.part + static_cast<int64_t>(blockIdx.x) * (a.n_in * a.n_out + a.n_out);
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int o = 0; o < OT; ++o) {
      const int in = 32 * i + (lane & 31);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int on = 32 * o + 8 * (r / 4) + 4 * h + r % 4;
        if (in < a.n_in && on < a.n_out) out[a.wb_by_out ? in * a.n_out + on : on * a.n_in + in] = wb[i][o][r];
      }
    }
  if ((lane & 31) == 0)
#pragma unroll
    for (int s = 0; s < SO; ++s)
#pragma unroll
      for (int k = 0; k < E; ++k)
        if ((2 * s + h) * E + k < a.n_out) out[a.n_in * a.n_out + (2 * s + h) * E + k] = bb[s][k];
#endif
}

// ---------------------------------------------------------------- launches

// As many workgroups as are resident (64 -> 64 bf16: four a CU, by LDS and by registers).  Fewer, so that every wave
// has the same number of tiles, leaves loads out at once: 214980 x 64 -> 64 bf16 22.8 us with 840 of 1024, 21.4 with
// all; 140000 x 17 -> 17 fp32 16.9 and 14.3; 500000 x 60 -> 31 bf16 34.3 and 35.3.
template <class T, int IT, int OT, bool kEven>
hipError_t launch_fwd(const FwdArgs& a, hipStream_t s) {
  static const int resident = [] {
    int n = 0;
    const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, fwd_kernel<T, IT, OT, kEven>, kFwdThreads, 0);
    return e == hipSuccess && n > 0 ? 256 * n : 256;
  }();
  const int64_t units = (static_cast<int64_t>(a.rows) + 32 * kFwdThreads / 64 - 1) / (32 * kFwdThreads / 64);
  const unsigned groups = static_cast<unsigned>(std::min<int64_t>(units, resident));
  fwd_kernel<T, IT, OT, kEven><<<dim3(groups), dim3(kFwdThreads), 0, s>>>(a);
  return hipGetLastError();
}
template <class T, int IT, int OT>
hipError_t launch_fwd(const FwdArgs& a, bool even, hipStream_t s) {
  return even ? launch_fwd<T, IT, OT, true>(a, s) : launch_fwd<T, IT, OT, false>(a, s);
}
template <class T, int IT, int OT>
hipError_t launch_bwd(const BwdArgs& a, bool even, int groups, hipStream_t s) {
  const dim3 grid(groups), block(bwd_threads<T>());
  if (a.z != nullptr) {
    if (even) bwd_kernel<T, IT, OT, true, true><<<grid, block, 0, s>>>(a);
    else bwd_kernel<T, IT, OT, false, true><<<grid, block, 0, s>>>(a);
  } else {
    if (even) bwd_kernel<T, IT, OT, true, false><<<grid, block, 0, s>>>(a);
    else bwd_kernel<T, IT, OT, false, false><<<grid, block, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t forward(const FwdArgs& a, bool even, hipStream_t s) {
  switch (tiles_of(a.n_in) * 8 + tiles_of(a.n_out)) {
    case 9: return launch_fwd<T, 1, 1>(a, even, s);
    case 10: return launch_fwd<T, 1, 2>(a, even, s);
    case 12: return launch_fwd<T, 1, 4>(a, even, s);
    case 17: return launch_fwd<T, 2, 1>(a, even, s);
    case 18: return launch_fwd<T, 2, 2>(a, even, s);
    case 20: return launch_fwd<T, 2, 4>(a, even, s);
    case 33: return launch_fwd<T, 4, 1>(a, even, s);
    default: return launch_fwd<T, 4, 2>(a, even, s);
  }
}
template <class T>
hipError_t backward(const BwdArgs& a, bool even, int groups, hipStream_t s) {
  switch (tiles_of(a.n_in) * 8 + tiles_of(a.n_out)) {
    case 9: return launch_bwd<T, 1, 1>(a, even, groups, s);
    case 10: return launch_bwd<T, 1, 2>(a, even, groups, s);
    case 17: return launch_bwd<T, 2, 1>(a, even, groups, s);
    case 18: return launch_bwd<T, 2, 2>(a, even, groups, s);
    default: return launch_bwd<T, 4, 1>(a, even, groups, s);
  }
}

}  // namespace narrow
}  // namespace etpc
