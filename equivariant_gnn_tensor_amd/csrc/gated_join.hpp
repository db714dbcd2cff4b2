// Row kernels of the gated residual join between two norms (templates; gated_join_*.hip hold
// the instantiations of one element type each).
//
//   xh = (x - mean) rstd,  n = xh w1 + b1,  p = 1 / (1 + exp(-gate)),  h = residual + scale p n,
//   hh = (h - mean_h) rstd_h,  y = hh w2 + b2
// and, with g2 = y_bar w2 and d = h_bar + rstd_h (g2 - mean(g2) - hh mean(g2 hh)), the gradient of h:
//   residual_bar = d,  u = d scale p,  gate_bar = u n (1 - p),
//   g1 = u w1,  x_bar = rstd (g1 - mean(g1) - xh mean(g1 xh)),
//   w1_bar = sum u xh, b1_bar = sum u, scale_bar = sum d p n, w2_bar = sum y_bar hh, b2_bar = sum y_bar.
//
// Memory bound, built like the layer norm (layer_norm.hpp): a group of G threads owns a row and
// keeps it in registers, so the sums of both norms cost no second read; statistics, sums and
// everything between load and store are fp32, and y comes from the unrounded h.
// Forward: 65408 x 1024 bf16, five rows moved for each (670 MB), 126 us, 5.3 TB/s, what a copy of that
// size reaches.  Backward: 4097 x 2047 fp32 (268 MB) 57 us, 4.7 TB/s, and 6.3 us for the second stage of
// the column sums.  Its five rows and five column sums a thread are the registers; above 4096 columns
// (a workgroup of 1024 to a row) four of the sums go to LDS: 8192 x 8192 bf16 243 us, 4.4 TB/s (549
// with the registers spilled), fp32 504 (919; 13 still spilled with a gate).  Forward rows of 8193 to 16384 columns
// spill 42 registers (fp32 with a gate), 16 (fp32), 14 and 10 (16 bits): 4096 x 16384 fp32 343 us, bf16 174, 3.9 TB/s.
#pragma once

#include "activation.hpp"
#include "gated_join_args.hpp"
#include "layer_norm.hpp"

namespace etpc {
namespace join {

using norm::Span;

// p = 1 / (1 + exp(-g)) and 1 - p, neither by a difference and from one exp that cannot overflow.
template <bool kWide>
__device__ inline void gate_pair(float g, float& p, float& q) {
  const float e = exp_of<kWide>(-1.f, fabsf(g)), r = inverse<kWide>(1.f + e), er = e * r;
  p = g >= 0.f ? r : er;
  q = g >= 0.f ? er : r;
}

// Mean and 1 / sqrt(variance + eps) of a row held as v[V][8]; v is centred on return.
template <int G, int kRows, int V, bool kEven>
__device__ inline void centre(float (&v)[V][8], const Span<G, V, kEven>& span, float inv_n, float cols, float eps,
                              float* lds, int& half, float& mean, float& rstd) {
  float s[1] = {0.f}, q[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += span.counts(i, k) ? v[i][k] : 0.f;
  group_sum<G, kRows>(s, lds, half);
  const float m = s[0] / cols;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[i][k] -= m;
      const float c = span.counts(i, k) ? v[i][k] : 0.f;
      q[0] = fmaf(c, c, q[0]);
      q[1] += c;
    }
  group_sum<G, kRows>(q, lds, half);
  const float off = q[1] * inv_n;
  rstd = norm_rstd(q[0], off, inv_n, eps);
  mean = norm_mean(m, off, rstd);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] -= off;
}

template <class T, int G, int V, bool kEven, bool kGate>
__global__ __launch_bounds__(norm::fwd_threads<G>()) void fwd_kernel(const JoinFwdArgs a) {
  constexpr int kRows = norm::fwd_threads<G>() / G;
  constexpr bool kWide = sizeof(T) == 4;
  constexpr bool kKeep = G < 512;   // the gains stay in registers; larger groups have none to spare
  __shared__ float lds[G > 64 ? 4 * G / 64 : 1];
  const Span<G, V, kEven> span(threadIdx.x % G, a.cols);
  const float inv_n = 1.f / static_cast<float>(a.cols), cols = static_cast<float>(a.cols);
  int half = 0;
  float wa[V][8], wb[V][8], w2[V][8], b2[V][8];   // scale w1, scale b1
  const auto first_gains = [&]() {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s[8];
      span.load_or(a.scale, i, 1.f, s);
      span.load_or(a.w1, i, 1.f, wa[i]);
      span.load_or(a.b1, i, 0.f, wb[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) wa[i][k] *= s[k], wb[i][k] *= s[k];
    }
  };
  const auto second_gains = [&]() {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      span.load_or(a.w2, i, 1.f, w2[i]);
      span.load_or(a.b2, i, 0.f, b2[i]);
    }
  };
  if (kKeep) first_gains(), second_gains();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + norm::group_index<G>(); row < a.rows; row += step) {
    float v[V][8];
    Vec8<T> gate[V], res[V];
#pragma unroll
    for (int i = 0; i < V; ++i) span.load(static_cast<const T*>(a.x) + row * a.xs, i, v[i]);
    if (kGate)
#pragma unroll
      for (int i = 0; i < V; ++i) gate[i] = span.fetch(static_cast<const T*>(a.gate) + row * a.gates, i);
    if (a.res != nullptr)
#pragma unroll
      for (int i = 0; i < V; ++i) res[i] = span.fetch(static_cast<const T*>(a.res) + row * a.ress, i);
    float st[4];
    centre<G, kRows>(v, span, inv_n, cols, a.eps, lds, half, st[0], st[1]);
    const float rstd = st[1];
    if (!kKeep) first_gains();
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] = fmaf(v[i][k] * rstd, wa[i][k], wb[i][k]);
        if (kGate) {
          float p, q;
          gate_pair<kWide>(static_cast<float>(gate[i][k]), p, q);
          v[i][k] *= p;
        }
      }
      if (a.res != nullptr)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] += static_cast<float>(res[i][k]);
      if (a.h != nullptr) span.store(static_cast<T*>(a.h) + row * a.hs, i, v[i]);
    }
    centre<G, kRows>(v, span, inv_n, cols, a.eps, lds, half, st[2], st[3]);
    if (a.stats != nullptr) __builtin_memcpy(a.stats + 4 * row, &st, sizeof(st));   // every thread, the same bits
    if (!kKeep) second_gains();
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = fmaf(v[i][k] * st[3], w2[i][k], b2[i][k]);
      span.store(static_cast<T*>(a.y) + row * a.ys, i, v[i]);
    }
  }
}

// ---------------------------------------------------------------- backward
// Threads of a workgroup: one shared between rows of up to a wave.
template <int G>
constexpr int bwd_threads() {
  return G > 64 ? G : 256;
}

template <class T, int G, bool kEven, bool kGate>
struct Row {
  Vec8<T> x, gate, h, y_bar, h_bar;
  VecN<float, 4> st;
  __device__ inline void read(const JoinBwdArgs& a, const Span<G, 1, kEven>& span, int64_t row) {
    __builtin_memcpy(&st, a.stats + 4 * row, sizeof(st));
    h = span.fetch(static_cast<const T*>(a.h) + row * a.hs, 0);
    y_bar = span.fetch(static_cast<const T*>(a.y_bar) + row * a.ybs, 0);
    if (a.h_bar != nullptr) h_bar = span.fetch(static_cast<const T*>(a.h_bar) + row * a.hbs, 0);
    x = span.fetch(static_cast<const T*>(a.x) + row * a.xs, 0);
    if (kGate) gate = span.fetch(static_cast<const T*>(a.gate) + row * a.gates, 0);
  }
};

// One vector a thread.  Each group walks its rows, fetches the next one's operands ahead and
// keeps its columns' five sums in registers (all but one in LDS where 1024 threads leave 128
// registers each); at the end the workgroup adds its groups in a fixed
// order and writes one row of `part`, [5][cols] (or the results, when it is the only workgroup).
template <class T, int G, bool kEven, bool kGate>
__global__ __launch_bounds__(bwd_threads<G>()) void bwd_kernel(const JoinBwdArgs a) {
  constexpr int kThreads = bwd_threads<G>(), kRows = kThreads / G;
  constexpr bool kWide = sizeof(T) == 4;
  constexpr bool kKeep = G < 1024, kAhead = G < 1024;   // 1024 threads leave 128 registers each
  constexpr int kReduce = G > 64 ? 4 * G / 64 : 0;
  constexpr bool kLdsSums = G >= 1024;
  __shared__ float lds[kReduce + (kRows > 1 ? 8 * kThreads : 1)];
  __shared__ float own[kLdsSums ? 4 * 8 * kThreads : 1];   // [sums 1 to 4][2][threads][4], each thread its own
  const int lane = threadIdx.x % G, group = threadIdx.x / G, n = a.cols;
  const Span<G, 1, kEven> span(lane, n);
  const float inv_n = 1.f / static_cast<float>(n);
  int half = 0;
  float w1[8], b1[8], sc[8], w2[8], sum[5][8] = {};
  const auto gains = [&]() {
    span.load_or(a.w1, 0, 1.f, w1);
    span.load_or(a.b1, 0, 0.f, b1);
    span.load_or(a.scale, 0, 1.f, sc);
  };
  if (kKeep) {
    gains();
    span.load_or(a.w2, 0, 1.f, w2);
  }
  const auto total = [&](int j, int k) -> float& {
    return kLdsSums && j > 0 ? own[(((j - 1) * 2 + k / 4) * kThreads + threadIdx.x) * 4 + k % 4] : sum[j][k];
  };
  if (kLdsSums)
#pragma unroll
    for (int i = 0; i < 32; ++i) total(1 + i / 8, i % 8) = 0.f;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + norm::group_index<G>();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  Row<T, G, kEven, kGate> next;
  if (kAhead && row < a.rows) next.read(a, span, row);
  for (; row < a.rows; row += step) {
    if (!kAhead) next.read(a, span, row);
    const Row<T, G, kEven, kGate> now = next;
    if (kAhead) next.read(a, span, row + step < a.rows ? row + step : row);
    if (!kKeep) span.load_or(a.w2, 0, 1.f, w2);
    float d[8], hh[8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float y = static_cast<float>(now.y_bar[k]);
      hh[k] = (static_cast<float>(now.h[k]) - now.st[2]) * now.st[3];
      float& s3 = total(3, k);
      s3 = fmaf(y, hh[k], s3);
      total(4, k) += y;
      d[k] = y * w2[k];
      const float c = span.counts(0, k) ? d[k] : 0.f;
      s[0] += c;
      s[1] = fmaf(c, hh[k], s[1]);
    }
    group_sum<G, kRows>(s, lds, half);
    const float h0 = s[0] * inv_n, h1 = s[1] * inv_n;
    if (!kKeep) gains();
    float xh[8], gb[8];
    s[0] = s[1] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      d[k] = now.st[3] * (d[k] - fmaf(hh[k], h1, h0));
      if (a.h_bar != nullptr) d[k] += static_cast<float>(now.h_bar[k]);
    }
    if (a.res_bar != nullptr) span.store(static_cast<T*>(a.res_bar) + row * a.rbs, 0, d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      xh[k] = (static_cast<float>(now.x[k]) - now.st[0]) * now.st[1];
      float p = 1.f, q = 0.f;
      if (kGate) gate_pair<kWide>(static_cast<float>(now.gate[k]), p, q);
      const float m = fmaf(xh[k], w1[k], b1[k]), dp = d[k] * p, u = dp * sc[k];
      gb[k] = u * m * q;
      float& s2 = total(2, k);
      s2 = fmaf(dp, m, s2);
      sum[0][k] = fmaf(u, xh[k], sum[0][k]);
      total(1, k) += u;
      d[k] = u * w1[k];
      const float c = span.counts(0, k) ? d[k] : 0.f;
      s[0] += c;
      s[1] = fmaf(c, xh[k], s[1]);
    }
    if (kGate && a.gate_bar != nullptr) span.store(static_cast<T*>(a.gate_bar) + row * a.gbs, 0, gb);
    if (a.x_bar == nullptr) continue;   // the same for every thread
    group_sum<G, kRows>(s, lds, half);
    const float x0 = s[0] * inv_n, x1 = s[1] * inv_n;
#pragma unroll
    for (int k = 0; k < 8; ++k) d[k] = now.st[1] * (d[k] - fmaf(xh[k], x1, x0));
    span.store(static_cast<T*>(a.x_bar) + row * a.xbs, 0, d);
  }
  if (!a.sums) return;
  if (kLdsSums)
#pragma unroll
    for (int i = 0; i < 32; ++i) sum[1 + i / 8][i % 8] = total(1 + i / 8, i % 8);
  const bool whole = gridDim.x == 1;
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    float* out = whole ? a.bar[j] : a.part + (static_cast<int64_t>(blockIdx.x) * 5 + j) * n;
    if (kRows == 1) {
      if (out != nullptr) span.store(out, 0, sum[j]);
    } else {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) lds[kReduce + (group * 8 + k) * G + lane] = sum[j][k];
      __syncthreads();
      for (int e = threadIdx.x; e < 8 * G; e += kThreads) {
        const Span<G, 1, kEven> of(e % G, n);
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < kRows; ++q) t += lds[kReduce + q * 8 * G + e];
        if (of.counts(0, e / G) && out != nullptr) out[of.at[0] + e / G] = t;
      }
    }
  }
}

// ---------------------------------------------------------------- rows that do not fit
// Longer rows are read again for each sum by a workgroup of 1024 threads.  The backward pass
// leaves each row's means of g2 and g2 hh (what d takes) for the column sums, which a launch of
// their own takes, a thread owning eight columns.
constexpr int kLong = 1024;

template <class T>
__device__ inline void load_row(const void* p, int64_t at, int c, int n, float missing, float (&v)[8]) {
  if (p != nullptr) {
    load<8, false>(static_cast<const T*>(p) + at, c, n, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = missing;
  }
}

// h of eight columns, given x's centred mean (mean and off) and rstd; zero past the row.
template <class T>
__device__ inline void long_h(const JoinFwdArgs& a, int64_t row, int c, float mean, float off, float rstd, float (&v)[8]) {
  float w[8], b[8], s[8], g[8], r[8];
  load<8, false>(static_cast<const T*>(a.x) + row * a.xs, c, a.cols, v);
  load_row<float>(a.w1, 0, c, a.cols, 1.f, w);
  load_row<float>(a.b1, 0, c, a.cols, 0.f, b);
  load_row<float>(a.scale, 0, c, a.cols, 1.f, s);
  load_row<T>(a.gate, row * a.gates, c, a.cols, 0.f, g);
  load_row<T>(a.res, row * a.ress, c, a.cols, 0.f, r);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float p = 1.f, q;
    if (a.gate != nullptr) gate_pair<sizeof(T) == 4>(g[k], p, q);
    v[k] = fmaf(((v[k] - mean) - off) * rstd, w[k] * s[k], b[k] * s[k]) * p + r[k];
  }
}

template <class T>
__global__ __launch_bounds__(kLong) void fwd_long_kernel(const JoinFwdArgs a) {
  __shared__ float lds[4 * kLong / 64];
  const int n = a.cols;
  const float inv_n = 1.f / static_cast<float>(n);
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float mean[2] = {0.f, 0.f}, off[2] = {0.f, 0.f}, rstd[2] = {1.f, 1.f};
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {   // the norm of x, then that of h
      const auto read = [&](int c, float (&v)[8]) {
        if (pass == 0) load<8, false>(static_cast<const T*>(a.x) + row * a.xs, c, n, v);
        else long_h<T>(a, row, c, mean[0], off[0], rstd[0], v);
      };
      float s[1] = {0.f}, q[2] = {0.f, 0.f};
      for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * kLong) {
        float v[8], t = 0.f;
        read(static_cast<int>(c), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) t += c + k < n ? v[k] : 0.f;
        s[0] += t;
      }
      group_sum<kLong, 1>(s, lds, half);
      mean[pass] = s[0] / static_cast<float>(n);
      for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * kLong) {
        float v[8], t0 = 0.f, t1 = 0.f;
        read(static_cast<int>(c), v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < n) {
            t0 = fmaf(v[k] - mean[pass], v[k] - mean[pass], t0);
            t1 += v[k] - mean[pass];
          }
        q[0] += t0;
        q[1] += t1;
      }
      group_sum<kLong, 1>(q, lds, half);
      off[pass] = q[1] * inv_n;
      rstd[pass] = norm_rstd(q[0], off[pass], inv_n, a.eps);
    }
    if (threadIdx.x == 0 && a.stats != nullptr) {
      const VecN<float, 4> st = {norm_mean(mean[0], off[0], rstd[0]), rstd[0], norm_mean(mean[1], off[1], rstd[1]),
                                 rstd[1]};
      __builtin_memcpy(a.stats + 4 * row, &st, sizeof(st));
    }
    for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
      const int c = static_cast<int>(cc);
      float v[8], w[8], b[8];
      long_h<T>(a, row, c, mean[0], off[0], rstd[0], v);
      if (a.h != nullptr) store<8, false>(static_cast<T*>(a.h) + row * a.hs, c, n, v);
      load_row<float>(a.w2, 0, c, n, 1.f, w);
      load_row<float>(a.b2, 0, c, n, 0.f, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(((v[k] - mean[1]) - off[1]) * rstd[1], w[k], b[k]);
      store<8, false>(static_cast<T*>(a.y) + row * a.ys, c, n, v);
    }
  }
}

// What the backward pass makes of eight columns of a row: d, then u and the rest from it.
struct Bars {
  float y[8], hh[8], d[8], xh[8], m[8], dp[8], u[8], gb[8];
};
template <class T>
__device__ inline void long_bars(const JoinBwdArgs& a, int64_t row, int c, const VecN<float, 4>& st, float h0, float h1,
                                 Bars& o) {
  const int n = a.cols;
  float h[8], hb[8], x[8], g[8], w1[8], b1[8], sc[8], w2[8];
  load<8, false>(static_cast<const T*>(a.h) + row * a.hs, c, n, h);
  load<8, false>(static_cast<const T*>(a.y_bar) + row * a.ybs, c, n, o.y);
  load_row<T>(a.h_bar, row * a.hbs, c, n, 0.f, hb);
  load<8, false>(static_cast<const T*>(a.x) + row * a.xs, c, n, x);
  load_row<T>(a.gate, row * a.gates, c, n, 0.f, g);
  load_row<float>(a.w1, 0, c, n, 1.f, w1);
  load_row<float>(a.b1, 0, c, n, 0.f, b1);
  load_row<float>(a.scale, 0, c, n, 1.f, sc);
  load_row<float>(a.w2, 0, c, n, 1.f, w2);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    o.hh[k] = (h[k] - st[2]) * st[3];
    o.d[k] = st[3] * (o.y[k] * w2[k] - fmaf(o.hh[k], h1, h0)) + hb[k];
    o.xh[k] = (x[k] - st[0]) * st[1];
    float p = 1.f, q = 0.f;
    if (a.gate != nullptr) gate_pair<sizeof(T) == 4>(g[k], p, q);
    o.m[k] = fmaf(o.xh[k], w1[k], b1[k]);
    o.dp[k] = o.d[k] * p;
    o.u[k] = o.dp[k] * sc[k];
    o.gb[k] = o.u[k] * o.m[k] * q;
  }
}

template <class T>
__global__ __launch_bounds__(kLong) void bwd_long_kernel(const JoinBwdArgs a) {
  __shared__ float lds[4 * kLong / 64];
  const int n = a.cols;
  const float inv_n = 1.f / static_cast<float>(n);
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    VecN<float, 4> st;
    __builtin_memcpy(&st, a.stats + 4 * row, sizeof(st));
    float s[2] = {0.f, 0.f};
    for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
      const int c = static_cast<int>(cc);
      float h[8], y[8], w[8], t0 = 0.f, t1 = 0.f;
      load<8, false>(static_cast<const T*>(a.h) + row * a.hs, c, n, h);
      load<8, false>(static_cast<const T*>(a.y_bar) + row * a.ybs, c, n, y);
      load_row<float>(a.w2, 0, c, n, 1.f, w);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < n) {
          t0 = fmaf(y[k], w[k], t0);
          t1 = fmaf(y[k] * w[k], (h[k] - st[2]) * st[3], t1);
        }
      s[0] += t0;
      s[1] += t1;
    }
    group_sum<kLong, 1>(s, lds, half);
    const float h0 = s[0] * inv_n, h1 = s[1] * inv_n;
    if (threadIdx.x == 0 && a.means != nullptr) a.means[2 * row] = h0, a.means[2 * row + 1] = h1;
    if (a.x_bar == nullptr && a.res_bar == nullptr && a.gate_bar == nullptr) continue;
    float x0 = 0.f, x1 = 0.f;
    if (a.x_bar != nullptr) {
      s[0] = s[1] = 0.f;
      for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
        const int c = static_cast<int>(cc);
        Bars o;
        float w[8], t0 = 0.f, t1 = 0.f;
        long_bars<T>(a, row, c, st, h0, h1, o);
        load_row<float>(a.w1, 0, c, n, 1.f, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < n) {
            t0 = fmaf(o.u[k], w[k], t0);
            t1 = fmaf(o.u[k] * w[k], o.xh[k], t1);
          }
        s[0] += t0;
        s[1] += t1;
      }
      group_sum<kLong, 1>(s, lds, half);
      x0 = s[0] * inv_n, x1 = s[1] * inv_n;
    }
    for (int64_t cc = 8 * threadIdx.x; cc < n; cc += 8 * kLong) {
      const int c = static_cast<int>(cc);
      Bars o;
      float w[8];
      long_bars<T>(a, row, c, st, h0, h1, o);
      if (a.res_bar != nullptr) store<8, false>(static_cast<T*>(a.res_bar) + row * a.rbs, c, n, o.d);
      if (a.gate_bar != nullptr) store<8, false>(static_cast<T*>(a.gate_bar) + row * a.gbs, c, n, o.gb);
      if (a.x_bar != nullptr) {
        load_row<float>(a.w1, 0, c, n, 1.f, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = st[1] * (o.u[k] * w[k] - fmaf(o.xh[k], x1, x0));
        store<8, false>(static_cast<T*>(a.x_bar) + row * a.xbs, c, n, w);
      }
    }
  }
}

template <class T>
__global__ __launch_bounds__(256) void bwd_long_cols_kernel(const JoinBwdArgs a) {
  const int n = a.cols;
  const int64_t cc = 8 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x);
  if (cc >= n) return;
  const int c = static_cast<int>(cc);
  float sum[5][8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    VecN<float, 4> st;
    __builtin_memcpy(&st, a.stats + 4 * row, sizeof(st));
    Bars o;
    long_bars<T>(a, row, c, st, a.means[2 * row], a.means[2 * row + 1], o);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sum[0][k] = fmaf(o.u[k], o.xh[k], sum[0][k]);
      sum[1][k] += o.u[k];
      sum[2][k] = fmaf(o.dp[k], o.m[k], sum[2][k]);
      sum[3][k] = fmaf(o.y[k], o.hh[k], sum[3][k]);
      sum[4][k] += o.y[k];
    }
  }
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    float* out = gridDim.y == 1 ? a.bar[j] : a.part + (static_cast<int64_t>(blockIdx.y) * 5 + j) * n;
    if (out != nullptr) store<8, false>(out, c, n, sum[j]);
  }
}

// ---------------------------------------------------------------- launches
constexpr int kFwdCols = norm::kRegCols, kBwdCols = 8192;   // longest rows kept in registers

template <class T, bool kEven, bool kGate>
struct LaunchFwd {
  const JoinFwdArgs& a;
  hipStream_t s;
  template <int G, int V>
  hipError_t operator()() const {
    constexpr int threads = norm::fwd_threads<G>(), rows = threads / G;
    const int64_t groups =
        std::min<int64_t>((static_cast<int64_t>(a.rows) + rows - 1) / rows, norm::fwd_waves<G, true>() / (threads / 64));
    fwd_kernel<T, G, V, kEven, kGate><<<dim3(static_cast<unsigned>(groups)), dim3(threads), 0, s>>>(a);
    return hipGetLastError();
  }
};

template <class T>
hipError_t launch_fwd(const JoinFwdArgs& a, hipStream_t s) {
  if (a.cols <= kFwdCols) {
    const bool even = a.cols % 8 == 0, gate = a.gate != nullptr;
    constexpr int size = sizeof(T);
    return even ? gate ? norm::fwd_shape<size>(a.cols, LaunchFwd<T, true, true>{a, s})
                       : norm::fwd_shape<size>(a.cols, LaunchFwd<T, true, false>{a, s})
           : gate ? norm::fwd_shape<size>(a.cols, LaunchFwd<T, false, true>{a, s})
                  : norm::fwd_shape<size>(a.cols, LaunchFwd<T, false, false>{a, s});
  }
  fwd_long_kernel<T><<<dim3(static_cast<unsigned>(std::min(a.rows, 2048))), dim3(kLong), 0, s>>>(a);
  return hipGetLastError();
}

// The smallest group that holds the row, one vector a thread.
template <class F>
auto bwd_shape(int32_t cols, F&& f) {
  if (cols <= 8) return f.template operator()<1>();
  if (cols <= 16) return f.template operator()<2>();
  if (cols <= 32) return f.template operator()<4>();
  if (cols <= 64) return f.template operator()<8>();
  if (cols <= 128) return f.template operator()<16>();
  if (cols <= 256) return f.template operator()<32>();
  if (cols <= 512) return f.template operator()<64>();
  if (cols <= 1024) return f.template operator()<128>();
  if (cols <= 2048) return f.template operator()<256>();
  if (cols <= 4096) return f.template operator()<512>();
  return f.template operator()<1024>();
}

template <class T, bool kEven, bool kGate>
struct LaunchBwd {
  const JoinBwdArgs& a;
  hipStream_t s;
  template <int G>
  hipError_t operator()() const {
    bwd_kernel<T, G, kEven, kGate><<<dim3(static_cast<unsigned>(a.parts)), dim3(bwd_threads<G>()), 0, s>>>(a);
    return hipGetLastError();
  }
};

template <class T>
hipError_t launch_bwd(const JoinBwdArgs& a, hipStream_t s) {
  if (a.cols <= kBwdCols) {
    const bool even = a.cols % 8 == 0, gate = a.gate != nullptr;
    return even ? gate ? bwd_shape(a.cols, LaunchBwd<T, true, true>{a, s}) : bwd_shape(a.cols, LaunchBwd<T, true, false>{a, s})
           : gate ? bwd_shape(a.cols, LaunchBwd<T, false, true>{a, s})
                  : bwd_shape(a.cols, LaunchBwd<T, false, false>{a, s});
  }
  bwd_long_kernel<T><<<dim3(static_cast<unsigned>(std::min(a.rows, 2048))), dim3(kLong), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.sums) return e;
  const int64_t vecs = (static_cast<int64_t>(a.cols) + 7) / 8;
  bwd_long_cols_kernel<T><<<dim3(static_cast<unsigned>((vecs + 255) / 256), static_cast<unsigned>(a.parts)), dim3(256), 0,
                           s>>>(a);
  return hipGetLastError();
}

hipError_t fwd_f32(const JoinFwdArgs& a, hipStream_t s);
hipError_t fwd_bf16(const JoinFwdArgs& a, hipStream_t s);
hipError_t fwd_f16(const JoinFwdArgs& a, hipStream_t s);
hipError_t bwd_f32(const JoinBwdArgs& a, hipStream_t s);
hipError_t bwd_bf16(const JoinBwdArgs& a, hipStream_t s);
hipError_t bwd_f16(const JoinBwdArgs& a, hipStream_t s);

}  // namespace join
}  // namespace etpc
