// Row kernels of the layer norm and its residual join (templates; layer_norm_*.hip hold the
// instantiations of one element type each).
//
//   h = res + dropout(x),  m = mean(h),  v = mean((h - m)^2),  r = 1 / sqrt(v + eps),
//   y = (h - m) r w + b
// and with xh = (h - m) r, g = y_bar w:
//   d = h_bar + r (g - mean(g) - xh mean(g xh)),  res_bar = d,  x_bar = dropout(d),
//   w_bar = sum_rows y_bar xh,  b_bar = sum_rows y_bar.
//
// Memory bound: one pass reads every operand once and writes every result once.  A group of
// G threads owns a row and keeps it in registers (8 V columns a thread), so the two sums of
// the forward pass (mean, then the sum of squares of what is left after it, which does not
// cancel) and the backward's two cost no second read.  Statistics, sums and the normalised
// row are fp32 whatever the element type; y comes from the unrounded h.
#pragma once

#include <algorithm>

#include "nodewise.hpp"
#include "rows.hpp"

namespace etpc {
namespace norm {

constexpr int kThreads = 256;
constexpr int kRegCols = 16384;   // longest row kept in registers: 512 threads of 32 columns

template <int G>
constexpr int threads_of() {
  return G > 64 ? G : kThreads;
}

template <class T, int G, int V, bool kEven>
__global__ __launch_bounds__(threads_of<G>()) void fwd_kernel(const NormFwdArgs a) {
  constexpr int kRows = threads_of<G>() / G;
  __shared__ float lds[G > 64 ? 2 * G / 64 : 1];
  const int lane = threadIdx.x % G, n = a.cols;
  const float inv_n = 1.f / static_cast<float>(n);
  const bool drop = a.drop.threshold != 0;
  const uint64_t offset = drop ? drop_offset(a.drop) : 0;
  int half = 0;
  float w[V][8], b[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 8 * (lane + i * G);
    if (a.w != nullptr) load<8, kEven>(a.w, c, n, w[i]);
    if (a.b != nullptr) load<8, kEven>(a.b, c, n, b[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (a.w == nullptr) w[i][k] = 1.f;
      if (a.b == nullptr) b[i][k] = 0.f;
    }
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) load<8, kEven>(x, 8 * (lane + i * G), n, v[i]);
    if (drop)
#pragma unroll
      for (int i = 0; i < V; ++i)
        drop8(v[i], philox(lane + i * G, static_cast<uint32_t>(row), offset, a.drop.seed), a.drop.threshold,
              a.drop.scale);
    if (a.res != nullptr) {
      const T* res = static_cast<const T*>(a.res) + row * a.ress;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float t[8];
        load<8, kEven>(res, 8 * (lane + i * G), n, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] += t[k];
      }
    }
    if (a.h != nullptr) {
      T* h = static_cast<T*>(a.h) + row * a.hs;
#pragma unroll
      for (int i = 0; i < V; ++i) store<8, kEven>(h, 8 * (lane + i * G), n, v[i]);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += v[i][k];
    group_sum<G>(s, lds, half);
    const float mean = s[0] / static_cast<float>(n);   // exact for a constant row, unlike s * (1 / n)
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] -= mean;
        if ((kEven ? 8 * (lane + i * G) : 8 * (lane + i * G) + k) < n) s[0] = fmaf(v[i][k], v[i][k], s[0]);
      }
    group_sum<G>(s, lds, half);
    const float rstd = 1.f / sqrtf(fmaf(s[0], inv_n, a.eps));
    if (lane == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ys;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = fmaf(v[i][k] * rstd, w[i][k], b[i][k]);
      store<8, kEven>(y, 8 * (lane + i * G), n, v[i]);
    }
  }
}

// Writes the gradient of one vector of columns, d + h_bar already added by the caller.
template <class T, bool kEven>
__device__ inline void store_bars(const NormBwdArgs& a, int64_t row, int c, float (&d)[8], bool drop, uint64_t offset) {
  if (a.res_bar != nullptr) store<8, kEven>(static_cast<T*>(a.res_bar) + row * a.rbs, c, a.cols, d);
  if (a.x_bar != nullptr) {
    if (drop)
      drop8(d, philox(c / 8, static_cast<uint32_t>(row), offset, a.drop.seed), a.drop.threshold, a.drop.scale);
    store<8, kEven>(static_cast<T*>(a.x_bar) + row * a.xbs, c, a.cols, d);
  }
}

// What the backward pass reads of one row, a thread's share.
template <class T, int G, int V, bool kEven>
struct Operands {
  Vec8<T> h[V], y_bar[V], h_bar[V];
  float mean, rstd;
  __device__ inline void read(const NormBwdArgs& a, int64_t row, int lane) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (lane + i * G);
      h[i] = fetch<8, kEven>(static_cast<const T*>(a.h) + row * a.hs, c, a.cols);
      y_bar[i] = fetch<8, kEven>(static_cast<const T*>(a.y_bar) + row * a.ybs, c, a.cols);
      if (a.h_bar != nullptr) h_bar[i] = fetch<8, kEven>(static_cast<const T*>(a.h_bar) + row * a.hbs, c, a.cols);
      else h_bar[i] = Vec8<T>{};
    }
    mean = a.mean[row];
    rstd = a.rstd[row];
  }
};

// Each group walks its rows and keeps its columns' sums of y_bar xh and y_bar; the next row's
// operands are fetched before this row's sums are taken.  At the end the workgroup adds its
// groups in a fixed order through LDS and writes one row of `part` (or the result itself,
// when it is the only workgroup).  One vector a thread: more threads a row measured faster
// than more registers a thread (8192 x 4096 fp16: 512 threads of one vector 54.6 us, 256 of
// two 81.4), the prefetch then gave 44.9.  Rows past 8192 columns need two vectors for 1024
// threads, whose sums then live in LDS (each thread its own places).
template <class T, int G, int V, bool kEven>
__global__ __launch_bounds__(threads_of<G>()) void bwd_kernel(const NormBwdArgs a) {
  constexpr int kRows = threads_of<G>() / G;
  constexpr bool kLdsSums = V > 1, kAhead = V * sizeof(T) <= 4;   // two f32 vectors of the next row would spill
  constexpr int kReduce = G > 64 ? 4 * G / 64 : 0;
  constexpr int kSums = kLdsSums ? 16 * V * G : kRows > 1 ? 16 * kThreads : 0;
  __shared__ float lds[kReduce + kSums];
  const int lane = threadIdx.x % G, group = threadIdx.x / G, n = a.cols;
  const float inv_n = 1.f / static_cast<float>(n);
  const bool drop = a.drop.threshold != 0, grads = a.x_bar != nullptr || a.res_bar != nullptr;
  const uint64_t offset = drop ? drop_offset(a.drop) : 0;
  int half = 0;
  float w[V][8], dw[kLdsSums ? 1 : V][8], db[kLdsSums ? 1 : V][8];
  float* own = lds + kReduce + threadIdx.x;   // with kLdsSums: sum k of vector i at own[(16 i + k) G]
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.w != nullptr) load<8, kEven>(a.w, 8 * (lane + i * G), n, w[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (a.w == nullptr) w[i][k] = 1.f;
      if (kLdsSums) own[(16 * i + k) * G] = own[(16 * i + 8 + k) * G] = 0.f;
      else dw[i][k] = db[i][k] = 0.f;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
  Operands<T, G, V, kEven> next;
  if (kAhead && row < a.rows) next.read(a, row, lane);
  for (; row < a.rows; row += step) {
    if (!kAhead) next.read(a, row, lane);
    const Operands<T, G, V, kEven> now = next;
    if (kAhead && row + step < a.rows) next.read(a, row + step, lane);
    float v[V][8], g[V][8], s[2] = {0.f, 0.f};
    // Columns past the row's end hold y_bar = 0, so they add nothing to any sum.
#pragma unroll
    for (int i = 0; i < V; ++i) {
      settle<8, kEven, T>(now.h[i], 8 * (lane + i * G), n, v[i]);
      settle<8, kEven, T>(now.y_bar[i], 8 * (lane + i * G), n, g[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] = (v[i][k] - now.mean) * now.rstd;
        if (kLdsSums) {
          own[(16 * i + k) * G] = fmaf(g[i][k], v[i][k], own[(16 * i + k) * G]);
          own[(16 * i + 8 + k) * G] += g[i][k];
        } else {
          dw[i][k] = fmaf(g[i][k], v[i][k], dw[i][k]);
          db[i][k] += g[i][k];
        }
        g[i][k] *= w[i][k];
        s[0] += g[i][k];
        s[1] = fmaf(g[i][k], v[i][k], s[1]);
      }
    }
    if (!grads) continue;
    group_sum<G>(s, lds, half);
    const float m0 = s[0] * inv_n, m1 = s[1] * inv_n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t[8];
      settle<8, kEven, T>(now.h_bar[i], 8 * (lane + i * G), n, t);
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] += now.rstd * (g[i][k] - fmaf(v[i][k], m1, m0));
      store_bars<T, kEven>(a, row, 8 * (lane + i * G), t, drop, offset);
    }
  }
  if (a.w_bar == nullptr && a.b_bar == nullptr) return;
  const bool whole = gridDim.x == 1;
  float* wo = whole ? a.w_bar : a.part + static_cast<int64_t>(blockIdx.x) * 2 * n;
  float* bo = whole ? a.b_bar : wo + n;
  if (kRows == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (kLdsSums)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dw[0][k] = own[(16 * i + k) * G];
          db[0][k] = own[(16 * i + 8 + k) * G];
        }
      if (wo != nullptr) store<8, kEven>(wo, 8 * (lane + i * G), n, dw[kLdsSums ? 0 : i]);
      if (bo != nullptr) store<8, kEven>(bo, 8 * (lane + i * G), n, db[kLdsSums ? 0 : i]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    lds[kReduce + (group * 8 + k) * G + lane] = dw[0][k];
    lds[kReduce + 8 * kThreads + (group * 8 + k) * G + lane] = db[0][k];
  }
  __syncthreads();
  for (int j = threadIdx.x; j < 16 * G; j += kThreads) {
    const int which = j / (8 * G), e = j % (8 * G), c = 8 * (e % G) + e / G;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kRows; ++q) t += lds[kReduce + which * 8 * kThreads + q * 8 * G + e];
    float* out = which ? bo : wo;
    if (c < n && out != nullptr) out[c] = t;
  }
}

// ---------------------------------------------------------------- rows that do not fit
// Longer rows are read again for each sum: a workgroup of 1024 threads owns a row, the
// second and third read come from L2 while the row fits it.
constexpr int kLong = 1024;

template <class T>
__device__ inline void long_h(const NormFwdArgs& a, int64_t row, int c, bool drop, uint64_t offset, float (&v)[8]) {
  load<8, false>(static_cast<const T*>(a.x) + row * a.xs, c, a.cols, v);
  if (drop)
    drop8(v, philox(c / 8, static_cast<uint32_t>(row), offset, a.drop.seed), a.drop.threshold, a.drop.scale);
  if (a.res != nullptr) {
    float t[8];
    load<8, false>(static_cast<const T*>(a.res) + row * a.ress, c, a.cols, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += t[k];
  }
}

template <class T>
__global__ __launch_bounds__(kLong) void fwd_long_kernel(const NormFwdArgs a) {
  __shared__ float lds[2 * kLong / 64];
  const int n = a.cols;
  const float inv_n = 1.f / static_cast<float>(n);
  const bool drop = a.drop.threshold != 0;
  const uint64_t offset = drop ? drop_offset(a.drop) : 0;
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s[1] = {0.f};
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * kLong) {
      float v[8], t = 0.f;
      long_h<T>(a, row, static_cast<int>(c), drop, offset, v);
      if (a.h != nullptr) store<8, false>(static_cast<T*>(a.h) + row * a.hs, static_cast<int>(c), n, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) t += v[k];
      s[0] += t;
    }
    group_sum<kLong>(s, lds, half);
    const float mean = s[0] / static_cast<float>(n);   // exact for a constant row, unlike s * (1 / n)
    s[0] = 0.f;
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * kLong) {
      float v[8], t = 0.f;
      long_h<T>(a, row, static_cast<int>(c), drop, offset, v);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < n) t = fmaf(v[k] - mean, v[k] - mean, t);
      s[0] += t;
    }
    group_sum<kLong>(s, lds, half);
    const float rstd = 1.f / sqrtf(fmaf(s[0], inv_n, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
      const int c = static_cast<int>(cc);
      float v[8], w[8], b[8];
      long_h<T>(a, row, c, drop, offset, v);
      if (a.w != nullptr) load<8, false>(a.w, c, n, w);
      if (a.b != nullptr) load<8, false>(a.b, c, n, b);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = fmaf((v[k] - mean) * rstd, a.w != nullptr ? w[k] : 1.f, a.b != nullptr ? b[k] : 0.f);
      store<8, false>(static_cast<T*>(a.y) + row * a.ys, c, n, v);
    }
  }
}

template <class T>
__global__ __launch_bounds__(kLong) void bwd_long_kernel(const NormBwdArgs a) {
  __shared__ float lds[4 * kLong / 64];
  const int n = a.cols;
  const float inv_n = 1.f / static_cast<float>(n);
  const bool drop = a.drop.threshold != 0;
  const uint64_t offset = drop ? drop_offset(a.drop) : 0;
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* h = static_cast<const T*>(a.h) + row * a.hs;
    const T* yb = static_cast<const T*>(a.y_bar) + row * a.ybs;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.f, 0.f};
    for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
      const int c = static_cast<int>(cc);
      float v[8], g[8], w[8], t0 = 0.f, t1 = 0.f;
      load<8, false>(h, c, n, v);
      load<8, false>(yb, c, n, g);
      if (a.w != nullptr) load<8, false>(a.w, c, n, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (a.w != nullptr) g[k] *= w[k];
        t0 += g[k];
        t1 = fmaf(g[k], (v[k] - mean) * rstd, t1);
      }
      s[0] += t0;
      s[1] += t1;
    }
    group_sum<kLong>(s, lds, half);
    const float m0 = s[0] * inv_n, m1 = s[1] * inv_n;
    for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
      const int c = static_cast<int>(cc);
      float v[8], g[8], w[8], t[8];
      load<8, false>(h, c, n, v);
      load<8, false>(yb, c, n, g);
      if (a.w != nullptr) load<8, false>(a.w, c, n, w);
      if (a.h_bar != nullptr) load<8, false>(static_cast<const T*>(a.h_bar) + row * a.hbs, c, n, t);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (a.w != nullptr) g[k] *= w[k];
        const float d = rstd * (g[k] - fmaf((v[k] - mean) * rstd, m1, m0));
        t[k] = a.h_bar != nullptr ? t[k] + d : d;
      }
      store_bars<T, false>(a, row, c, t, drop, offset);
    }
  }
}

// Column sums of the long rows: a thread owns eight columns, blockIdx.y a slice of the rows.
template <class T>
__global__ __launch_bounds__(kThreads) void bwd_long_cols_kernel(const NormBwdArgs a) {
  const int n = a.cols;
  const int64_t cc = 8 * (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x);
  if (cc >= n) return;
  const int c = static_cast<int>(cc);
  float dw[8] = {}, db[8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float v[8], g[8];
    load<8, false>(static_cast<const T*>(a.h) + row * a.hs, c, n, v);
    load<8, false>(static_cast<const T*>(a.y_bar) + row * a.ybs, c, n, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      dw[k] = fmaf(g[k], (v[k] - mean) * rstd, dw[k]);
      db[k] += g[k];
    }
  }
  const bool whole = gridDim.y == 1;
  float* wo = whole ? a.w_bar : a.part + static_cast<int64_t>(blockIdx.y) * 2 * n;
  float* bo = whole ? a.b_bar : wo + n;
  if (wo != nullptr) store<8, false>(wo, c, n, dw);
  if (bo != nullptr) store<8, false>(bo, c, n, db);
}

// ---------------------------------------------------------------- launch shapes
// Threads per row and vectors of eight columns per thread, from the row length alone: the
// smallest group that holds the row, up to one wave with one vector; then more vectors
// (rows to 2048 columns stay within one wave: no barrier), then several waves.
template <class F>
auto by_cols_bwd(int32_t cols, F&& f) {
  if (cols <= 8) return f.template operator()<1, 1>();
  if (cols <= 16) return f.template operator()<2, 1>();
  if (cols <= 32) return f.template operator()<4, 1>();
  if (cols <= 64) return f.template operator()<8, 1>();
  if (cols <= 128) return f.template operator()<16, 1>();
  if (cols <= 256) return f.template operator()<32, 1>();
  if (cols <= 512) return f.template operator()<64, 1>();
  if (cols <= 1024) return f.template operator()<128, 1>();
  if (cols <= 2048) return f.template operator()<256, 1>();
  if (cols <= 4096) return f.template operator()<512, 1>();
  if (cols <= 8192) return f.template operator()<1024, 1>();
  return f.template operator()<1024, 2>();
}

template <class F>
auto by_cols(int32_t cols, F&& f) {
  if (cols <= 8) return f.template operator()<1, 1>();
  if (cols <= 16) return f.template operator()<2, 1>();
  if (cols <= 32) return f.template operator()<4, 1>();
  if (cols <= 64) return f.template operator()<8, 1>();
  if (cols <= 128) return f.template operator()<16, 1>();
  if (cols <= 256) return f.template operator()<32, 1>();
  if (cols <= 512) return f.template operator()<64, 1>();
  if (cols <= 1024) return f.template operator()<64, 2>();
  if (cols <= 2048) return f.template operator()<64, 4>();
  if (cols <= 4096) return f.template operator()<256, 2>();
  if (cols <= 8192) return f.template operator()<256, 4>();
  return f.template operator()<512, 4>();
}

constexpr int kFwdGroups = 2048;

template <class T, bool kEven>
struct LaunchFwd {
  const NormFwdArgs& a;
  hipStream_t s;
  template <int G, int V>
  hipError_t operator()() const {
    constexpr int threads = threads_of<G>(), rows = threads / G;
    const int64_t groups = std::min<int64_t>((static_cast<int64_t>(a.rows) + rows - 1) / rows, kFwdGroups);
    fwd_kernel<T, G, V, kEven><<<dim3(static_cast<unsigned>(groups)), dim3(threads), 0, s>>>(a);
    return hipGetLastError();
  }
};

template <class T, bool kEven>
struct LaunchBwd {
  const NormBwdArgs& a;
  hipStream_t s;
  template <int G, int V>
  hipError_t operator()() const {
    bwd_kernel<T, G, V, kEven><<<dim3(static_cast<unsigned>(norm_parts(a.rows, a.cols))), dim3(threads_of<G>()), 0, s>>>(a);
    return hipGetLastError();
  }
};

template <class T>
hipError_t launch_fwd(const NormFwdArgs& a, hipStream_t s) {
  if (a.cols <= kRegCols)
    return a.cols % 8 == 0 ? by_cols(a.cols, LaunchFwd<T, true>{a, s}) : by_cols(a.cols, LaunchFwd<T, false>{a, s});
  fwd_long_kernel<T><<<dim3(static_cast<unsigned>(std::min(a.rows, kFwdGroups))), dim3(kLong), 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.cols <= kRegCols)
    return a.cols % 8 == 0 ? by_cols_bwd(a.cols, LaunchBwd<T, true>{a, s})
                           : by_cols_bwd(a.cols, LaunchBwd<T, false>{a, s});
  if (a.x_bar != nullptr || a.res_bar != nullptr) {
    bwd_long_kernel<T><<<dim3(static_cast<unsigned>(std::min(a.rows, kFwdGroups))), dim3(kLong), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.w_bar == nullptr && a.b_bar == nullptr) return hipSuccess;
  const int64_t vecs = (static_cast<int64_t>(a.cols) + 7) / 8;
  bwd_long_cols_kernel<T><<<dim3(static_cast<unsigned>((vecs + kThreads - 1) / kThreads),
                                static_cast<unsigned>(norm_parts(a.rows, a.cols))),
                           dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

#define ETPC_NORM_TYPE(T, name)                                                                       \
  hipError_t fwd_##name(const NormFwdArgs& a, hipStream_t s) { return launch_fwd<T>(a, s); }          \
  hipError_t bwd_##name(const NormBwdArgs& a, hipStream_t s) { return launch_bwd<T>(a, s); }

hipError_t fwd_f32(const NormFwdArgs& a, hipStream_t s);
hipError_t fwd_bf16(const NormFwdArgs& a, hipStream_t s);
hipError_t fwd_f16(const NormFwdArgs& a, hipStream_t s);
hipError_t bwd_f32(const NormBwdArgs& a, hipStream_t s);
hipError_t bwd_bf16(const NormBwdArgs& a, hipStream_t s);
hipError_t bwd_f16(const NormBwdArgs& a, hipStream_t s);

}  // namespace norm
}  // namespace etpc
