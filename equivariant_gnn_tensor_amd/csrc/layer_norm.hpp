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
// G threads owns a row and keeps it in registers (8 V columns a thread), so the sums of the
// forward pass (mean, then sum and sum of squares of what is left after it, which do not
// cancel; the sum is what the rounded mean is off by, and corrects it) and the backward's two
// cost no second read.  Statistics, sums and the normalised row are fp32 whatever the element
// type; y comes from the unrounded h.
#pragma once

#include <algorithm>

#include "nodewise.hpp"
#include "rows.hpp"

namespace etpc {
namespace norm {

constexpr int kThreads = 256;
constexpr int kRegCols = 16384;   // longest row kept in registers

// Threads of a workgroup: the forward pass shares one between rows of up to a wave, the
// backward pass also between two rows of two waves (fewer rows of partial sums).
template <int G>
constexpr int fwd_threads() {
  return G > 64 ? G : kThreads;
}
template <int G>
constexpr int bwd_threads() {
  return G > 128 ? G : kThreads;
}

// Both by value, so that the arrays they come from stay in registers.
__device__ inline uint32_t pick(bool c, uint32_t a, uint32_t b) { return c ? a : b; }

// Where a thread's vector i lies in a row of n columns.  A vector that would start or end
// past the row is moved back to the row's last eight columns: every access is one full
// vector inside the row, with no branch around it, and what it holds and writes there is
// bit for bit what the columns' owners hold and write.  Only sums tell the copies apart:
// element k counts from `skip` on (8: a copy as a whole).  Rows shorter than a vector (one
// thread each) are read and written by elements.
template <int G, int V, bool kEven>
struct Span {
  int n, at[V], skip[V];
  __device__ inline Span(int lane, int cols) : n(cols) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (lane + i * G);
      at[i] = tiny() ? 0 : min(c, n - 8);
      skip[i] = tiny() ? 0 : min(c - at[i], 8);
    }
  }
  __device__ inline bool tiny() const { return G == 1 && !kEven && n < 8; }
  __device__ inline bool counts(int i, int k) const {
    return kEven ? skip[i] == 0 : k >= skip[i] && (G > 1 || k < n);
  }
  template <class T>
  __device__ inline Vec8<T> fetch(const T* __restrict__ row, int i) const {
    Vec8<T> t = {};
    if (tiny()) {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < n) t[k] = row[k];
    } else {
      __builtin_memcpy(&t, row + static_cast<unsigned>(at[i]), sizeof(t));
    }
    return t;
  }
  template <class T>
  __device__ inline void load(const T* __restrict__ row, int i, float (&v)[8]) const {
    const Vec8<T> t = fetch(row, i);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(t[k]);
  }
  template <class T>
  __device__ inline void load_or(const T* __restrict__ row, int i, float missing, float (&v)[8]) const {
    if (row != nullptr) {
      load(row, i, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = missing;
    }
  }
  // Rounds to the element type here, once (to nearest, ties to even).
  template <class T>
  __device__ inline void store(T* __restrict__ row, int i, const float (&v)[8]) const {
    Vec8<T> t;
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = static_cast<T>(v[k]);
    if (tiny()) {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < n) row[k] = t[k];
    } else {
      __builtin_memcpy(row + static_cast<unsigned>(at[i]), &t, sizeof(t));
    }
  }
  // The mask of a vector that was moved back takes its fields from two generator calls.
  __device__ inline void drop(float (&v)[8], int i, int64_t row, uint64_t offset, const DropArgs& d) const {
    Philox r = philox(static_cast<uint32_t>(at[i]) / 8, static_cast<uint32_t>(row), offset, d.seed);
    const int by = kEven ? 0 : at[i] % 8;
    if (by != 0) {
      const Philox q = philox(static_cast<uint32_t>(at[i]) / 8 + 1, static_cast<uint32_t>(row), offset, d.seed);
      const uint32_t w[8] = {r.w[0], r.w[1], r.w[2], r.w[3], q.w[0], q.w[1], q.w[2], q.w[3]};
      uint32_t by4[6], by2[5];
#pragma unroll
      for (int k = 0; k < 6; ++k) by4[k] = pick(by & 4, w[k + 2], w[k]);
#pragma unroll
      for (int k = 0; k < 5; ++k) by2[k] = pick(by & 2, by4[k + 1], by4[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[k] = pick(by & 1, (by2[k] >> 16) | (by2[k + 1] << 16), by2[k]);
    }
    drop8(v, r, d.threshold, d.scale);
  }
};

// The row of a thread's group among the kRows of its workgroup; rows of whole waves get it in
// a scalar register.
template <int G>
__device__ inline int group_index() {
  const int group = threadIdx.x / G;
  return G >= 64 ? __builtin_amdgcn_readfirstlane(group) : group;
}

// Read and write one row after another, no prefetch: waves enough are in flight, and fetching
// a row ahead measured slower (65536 x 512 bf16 24.8 us without, 28 to 30 with).
// What it reaches (reads and writes): 65536 x 512 bf16 23.2 us, 5.8 TB/s; 8192 x 2048 fp32
// 26.4 us, 5.1 TB/s; join 65408 x 1024 bf16 98.6 us, 5.4 TB/s.  A copy of the same bytes runs
// at 5.5, 5.5 and 5.4.
template <class T, int G, int V, bool kEven, bool kJoin>
__global__ __launch_bounds__(fwd_threads<G>()) void fwd_kernel(const NormFwdArgs a) {
  constexpr int kRows = fwd_threads<G>() / G;
  __shared__ float lds[G > 64 ? 4 * G / 64 : 1];
  const Span<G, V, kEven> span(threadIdx.x % G, a.cols);
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const bool drop = kJoin && a.drop.threshold != 0;
  const uint64_t offset = drop ? drop_offset(a.drop) : 0;
  int half = 0;
  float w[V][8], b[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    span.load_or(a.w, i, 1.f, w[i]);
    span.load_or(a.b, i, 0.f, b[i]);
  }
  // Adjacent rows go to adjacent groups: the rows in flight are one window of memory (equal
  // shares of adjacent rows measured 5 to 15 % slower).
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group_index<G>(); row < a.rows; row += step) {
    float v[V][8], s[1] = {0.f}, q[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) span.load(static_cast<const T*>(a.x) + row * a.xs, i, v[i]);
    if (kJoin) {
      Vec8<T> res[V];
      if (a.res != nullptr)
#pragma unroll
        for (int i = 0; i < V; ++i) res[i] = span.fetch(static_cast<const T*>(a.res) + row * a.ress, i);
      if (drop)
#pragma unroll
        for (int i = 0; i < V; ++i) span.drop(v[i], i, row, offset, a.drop);
      if (a.res != nullptr)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] += static_cast<float>(res[i][k]);
      if (a.h != nullptr)
#pragma unroll
        for (int i = 0; i < V; ++i) span.store(static_cast<T*>(a.h) + row * a.hs, i, v[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += span.counts(i, k) ? v[i][k] : 0.f;
    group_sum<G, kRows>(s, lds, half);
    const float mean = s[0] / static_cast<float>(a.cols);   // one rounding, s * (1 / n) has two
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] -= mean;
        const float c = span.counts(i, k) ? v[i][k] : 0.f;
        q[0] = fmaf(c, c, q[0]);
        q[1] += c;
      }
    group_sum<G, kRows>(q, lds, half);
    const float off = q[1] * inv_n, rstd = norm_rstd(q[0], off, inv_n, a.eps);
    if (a.mean != nullptr) a.mean[row] = norm_mean(mean, off, rstd);   // every thread of the group, the same bits
    if (a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = fmaf((v[i][k] - off) * rstd, w[i][k], b[i][k]);
      span.store(static_cast<T*>(a.y) + row * a.ys, i, v[i]);
    }
  }
}

// Eight elements on their way into registers.  A 16-byte load of 16-bit elements whose
// address is odd in elements takes about three cycles a lane, so two streams of them bound the
// backward pass of long rows (32768 rows of 2047 bf16: 104 us).  With kOdd such a vector is
// read one element lower, or one higher where it starts the row, and its eighth element on
// its own: everything stays inside the row, which has nine elements at least (83 us; rows up
// to 1024 columns gain nothing: 100000 x 65 13.8 -> 15.1).
template <class T, bool kOdd>
struct Raw8 {
  Vec8<T> t;
  T extra;
  int shift;   // 0: t is the vector; -1, 1: t lies one element lower, higher
  __device__ inline void read(const T* __restrict__ p, bool first) {
    shift = (reinterpret_cast<uintptr_t>(p) & 2) == 0 ? 0 : first ? 1 : -1;
    __builtin_memcpy(&t, __builtin_assume_aligned(p + shift, 4), sizeof(t));
    extra = p[shift < 0 ? 7 : 0];
  }
  __device__ inline Vec8<T> get() const {
    uint32_t d[4], o[4];
    uint16_t e;
    __builtin_memcpy(d, &t, sizeof(d));
    __builtin_memcpy(&e, &extra, sizeof(e));
    const uint32_t s[5] = {pick(shift > 0, static_cast<uint32_t>(e) << 16, d[0]), pick(shift > 0, d[0], d[1]),
                           pick(shift > 0, d[1], d[2]), pick(shift > 0, d[2], d[3]), pick(shift > 0, d[3], e)};
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = pick(shift != 0, (s[k] >> 16) | (s[k + 1] << 16), d[k]);
    Vec8<T> v;
    __builtin_memcpy(&v, o, sizeof(v));
    return v;
  }
};
template <class T>
struct Raw8<T, false> {
  Vec8<T> t;
  __device__ inline Vec8<T> get() const { return t; }
};

// What the backward pass reads of one row, a thread's share.
template <class T, int G, int V, bool kEven, bool kJoin, bool kOdd>
struct Operands {
  Raw8<T, kOdd> h[V], y_bar[V], h_bar[kJoin ? V : 1];
  float mean, rstd;
  __device__ inline void one(Raw8<T, kOdd>& r, const Span<G, V, kEven>& span, const void* p, int64_t at, int i) {
    if constexpr (kOdd) r.read(static_cast<const T*>(p) + at + span.at[i], span.at[i] == 0);
    else r.t = span.fetch(static_cast<const T*>(p) + at, i);
  }
  __device__ inline void read(const NormBwdArgs& a, const Span<G, V, kEven>& span, int64_t row) {
    if (kJoin && a.h_bar != nullptr)
#pragma unroll
      for (int i = 0; i < V; ++i) one(h_bar[i], span, a.h_bar, row * a.hbs, i);
    mean = a.mean[row];
    rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      one(h[i], span, a.h, row * a.hs, i);
      one(y_bar[i], span, a.y_bar, row * a.ybs, i);
    }
  }
};

// Each group walks its rows and keeps its columns' sums of y_bar xh and y_bar; the next row's
// operands are fetched before this row's sums are taken.  At the end the workgroup adds its
// groups in a fixed order through LDS and writes one row of `part` (or the result itself,
// when it is the only workgroup).  One vector a thread: more threads a row measured faster
// than more registers a thread (8192 x 4096 fp16: 512 threads of one vector 54.6 us, 256 of
// two 81.4), the prefetch then gave 44.9.  Rows past 8192 columns need two vectors for 1024
// threads, whose sums then live in LDS (each thread its own places).
// What it reaches, sums included: 8192 x 4096 fp16 43.2 us, 4.7 TB/s; 65536 x 512 bf16
// 41.0 us, 4.9 TB/s; join 65408 x 1024 bf16 131 us, 5.1 TB/s; 32768 x 2047 bf16 83 us, 4.9 TB/s.
template <class T, int G, int V, bool kEven, bool kJoin, bool kOdd>
__global__ __launch_bounds__(bwd_threads<G>()) void bwd_kernel(const NormBwdArgs a) {
  constexpr int kRows = bwd_threads<G>() / G;
  constexpr bool kBarrier = G > 64 && kRows > 1;   // rows that share a barrier take it together
  constexpr bool kLdsSums = V > 1, kAhead = V * sizeof(T) <= 4;   // two f32 vectors of the next row would spill
  constexpr int kReduce = G > 64 ? 4 * bwd_threads<G>() / 64 : 0;
  constexpr int kSums = kLdsSums ? 16 * V * G : kRows > 1 ? 16 * kThreads : 0;
  __shared__ float lds[kReduce + kSums];
  const int lane = threadIdx.x % G, group = threadIdx.x / G, n = a.cols;
  const Span<G, V, kEven> span(lane, n);
  const float inv_n = 1.f / static_cast<float>(n);
  const bool drop = kJoin && a.drop.threshold != 0, grads = a.x_bar != nullptr || (kJoin && a.res_bar != nullptr);
  const uint64_t offset = drop ? drop_offset(a.drop) : 0;
  int half = 0;
  float w[V][8], dw[kLdsSums ? 1 : V][8], db[kLdsSums ? 1 : V][8];
  float* own = lds + kReduce + threadIdx.x;   // with kLdsSums: sum k of vector i at own[(16 i + k) G]
#pragma unroll
  for (int i = 0; i < V; ++i) {
    span.load_or(a.w, i, 1.f, w[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (kLdsSums) own[(16 * i + k) * G] = own[(16 * i + 8 + k) * G] = 0.f;
      else dw[i][k] = db[i][k] = 0.f;
    }
  }
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group_index<G>();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  Operands<T, G, V, kEven, kJoin, kOdd> next;
  if (kAhead && row < a.rows) next.read(a, span, row);
  for (; kBarrier ? row - group_index<G>() < a.rows : row < a.rows; row += step) {
    if (kBarrier && row >= a.rows) {   // the last step may have a row for the first group only
      float none[2] = {0.f, 0.f};
      if (grads) group_sum<G, kRows>(none, lds, half);
      continue;
    }
    if (!kAhead) next.read(a, span, row);
    const Operands<T, G, V, kEven, kJoin, kOdd> now = next;
    if (kAhead) next.read(a, span, row + step < a.rows ? row + step : row);
    float v[V][8], g[V][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Vec8<T> h = now.h[i].get(), y_bar = now.y_bar[i].get();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float y = static_cast<float>(y_bar[k]);
        v[i][k] = (static_cast<float>(h[k]) - now.mean) * now.rstd;
        if (kLdsSums) {
          own[(16 * i + k) * G] = fmaf(y, v[i][k], own[(16 * i + k) * G]);
          own[(16 * i + 8 + k) * G] += y;
        } else {
          dw[i][k] = fmaf(y, v[i][k], dw[i][k]);
          db[i][k] += y;
        }
        g[i][k] = y * w[i][k];
        const float c = span.counts(i, k) ? g[i][k] : 0.f;
        s[0] += c;
        s[1] = fmaf(c, v[i][k], s[1]);
      }
    }
    if (!grads) continue;
    group_sum<G, kRows>(s, lds, half);
    const float m0 = s[0] * inv_n, m1 = s[1] * inv_n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = now.rstd * (g[i][k] - fmaf(v[i][k], m1, m0));
      if (kJoin && a.h_bar != nullptr) {
        const Vec8<T> h_bar = now.h_bar[i].get();
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] += static_cast<float>(h_bar[k]);
      }
      if (kJoin) {
        if (a.res_bar != nullptr) span.store(static_cast<T*>(a.res_bar) + row * a.rbs, i, t);
        if (drop) span.drop(t, i, row, offset, a.drop);
      }
      if (!kJoin || a.x_bar != nullptr) span.store(static_cast<T*>(a.x_bar) + row * a.xbs, i, t);
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
      if (wo != nullptr) span.store(wo, i, dw[kLdsSums ? 0 : i]);
      if (bo != nullptr) span.store(bo, i, db[kLdsSums ? 0 : i]);
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
    const int which = j / (8 * G), e = j % (8 * G);
    const Span<G, 1, kEven> of(e % G, n);
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kRows; ++q) t += lds[kReduce + which * 8 * kThreads + q * 8 * G + e];
    float* out = which ? bo : wo;
    if (of.counts(0, e / G) && out != nullptr) out[of.at[0] + e / G] = t;
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
  __shared__ float lds[4 * kLong / 64];
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
    group_sum<kLong, 1>(s, lds, half);
    const float mean = s[0] / static_cast<float>(n);   // one rounding, s * (1 / n) has two
    float q[2] = {0.f, 0.f};
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * kLong) {
      float v[8], t0 = 0.f, t1 = 0.f;
      long_h<T>(a, row, static_cast<int>(c), drop, offset, v);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < n) {
          t0 = fmaf(v[k] - mean, v[k] - mean, t0);
          t1 += v[k] - mean;
        }
      q[0] += t0;
      q[1] += t1;
    }
    group_sum<kLong, 1>(q, lds, half);
    const float off = q[1] * inv_n, rstd = norm_rstd(q[0], off, inv_n, a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = norm_mean(mean, off, rstd);
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
        v[k] = fmaf(((v[k] - mean) - off) * rstd, a.w != nullptr ? w[k] : 1.f, a.b != nullptr ? b[k] : 0.f);
      store<8, false>(static_cast<T*>(a.y) + row * a.ys, c, n, v);
    }
  }
}

// Writes the gradient of one vector of columns.
template <class T>
__device__ inline void store_bars(const NormBwdArgs& a, int64_t row, int c, float (&d)[8], bool drop, uint64_t offset) {
  if (a.res_bar != nullptr) store<8, false>(static_cast<T*>(a.res_bar) + row * a.rbs, c, a.cols, d);
  if (a.x_bar != nullptr) {
    if (drop)
      drop8(d, philox(c / 8, static_cast<uint32_t>(row), offset, a.drop.seed), a.drop.threshold, a.drop.scale);
    store<8, false>(static_cast<T*>(a.x_bar) + row * a.xbs, c, a.cols, d);
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
    group_sum<kLong, 1>(s, lds, half);
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
      store_bars<T>(a, row, c, t, drop, offset);
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
// Threads per row and vectors of eight columns per thread, from the row length and the
// element size: the smallest group that holds the row.  Forward, 16-bit rows past 64 columns
// take two vectors a thread (32768 x 1024 bf16: 24.3 us with two, 28.9 with one, 25.7 with
// four; 8192 x 4096 fp16: 26.0 with two, 30.5 with one, 28.6 with four), fp32 rows past 512
// (one and two are level, two halves the waves at a barrier: 8192 x 2048 26.4 us with two,
// 26.5 with one, 27.6 with four; 4096 x 4096 25.7, 26.6, 27.6; 16384 x 1024 27.0, 25.6, 27.1).
template <int kSize, class F>
auto fwd_shape(int32_t cols, F&& f) {
  if (cols <= 8) return f.template operator()<1, 1>();
  if (cols <= 16) return f.template operator()<2, 1>();
  if (cols <= 32) return f.template operator()<4, 1>();
  if (cols <= 64) return f.template operator()<8, 1>();
  if constexpr (kSize == 2) {
    if (cols <= 128) return f.template operator()<8, 2>();
    if (cols <= 256) return f.template operator()<16, 2>();
    if (cols <= 512) return f.template operator()<32, 2>();
    if (cols <= 1024) return f.template operator()<64, 2>();
    if (cols <= 2048) return f.template operator()<128, 2>();
    if (cols <= 4096) return f.template operator()<256, 2>();
    if (cols <= 8192) return f.template operator()<512, 2>();
    return f.template operator()<1024, 2>();
  }
  if (cols <= 128) return f.template operator()<16, 1>();
  if (cols <= 256) return f.template operator()<32, 1>();
  if (cols <= 512) return f.template operator()<64, 1>();
  if (cols <= 1024) return f.template operator()<64, 2>();
  if (cols <= 2048) return f.template operator()<128, 2>();
  if (cols <= 4096) return f.template operator()<256, 2>();
  if (cols <= 8192) return f.template operator()<512, 2>();
  return f.template operator()<1024, 2>();
}

// Backward: one vector a thread, except past 8192 columns.  Between 4096 and 8192 also 640 and
// 768 threads (6710 x 5000 bf16: 43.9 us with 640, 53.6 with 1024); 192 and 384 threads
// measured slower than 256 and 512 with idle lanes (6553 x 2560 fp32: 50.1 us against 42.9).
template <class F>
auto bwd_shape(int32_t cols, F&& f) {
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
  if (cols <= 5120) return f.template operator()<640, 1>();
  if (cols <= 6144) return f.template operator()<768, 1>();
  if (cols <= 8192) return f.template operator()<1024, 1>();
  return f.template operator()<1024, 2>();
}

// Workgroups of the forward pass by waves a CU.  Where a barrier ties waves together, as many
// as are resident at once (8192 x 4096 fp16: 25.1 us with 24, 28.1 with 32, 27.4 with 64).
// Otherwise 64, more than fit, so that a CU whose rows are done takes others (100000 x 256
// bf16: 17.3 us with 64, 18.1 with 32, 18.4 with 24; the join of 8192 x 4096 bf16: 50.6 with
// 64, 52.7 with 32, 53.4 with 24).  Groups of up to 8 lanes, 64 against 32: 400000 x 128 bf16
// 38.4 and 41.0 us, 400000 x 32 fp32 18.0 and 19.1, 214980 x 64 bf16 11.0 and 11.1, 65408 x 64
// fp32 of rows of 576 8.1 and 8.1, the join of 214980 x 128 bf16 41.4 and 44.4; 32 is the
// faster for 100000 x 64 fp32 (10.8 and 10.1) and rows of 8 (1000000 fp32 13.6 and 12.5).
template <int G, bool kJoin>
constexpr int fwd_waves() {
  return 256 * (G <= 64 || kJoin ? 64 : G < 1024 ? 24 : 32);
}

template <class T, bool kEven, bool kJoin>
struct LaunchFwd {
  const NormFwdArgs& a;
  hipStream_t s;
  template <int G, int V>
  hipError_t operator()() const {
    constexpr int threads = fwd_threads<G>(), rows = threads / G;
    const int64_t groups =
        std::min<int64_t>((static_cast<int64_t>(a.rows) + rows - 1) / rows, fwd_waves<G, kJoin>() / (threads / 64));
    fwd_kernel<T, G, V, kEven, kJoin><<<dim3(static_cast<unsigned>(groups)), dim3(threads), 0, s>>>(a);
    return hipGetLastError();
  }
};

template <class T, bool kEven, bool kJoin, bool kOdd>
struct LaunchBwd {
  const NormBwdArgs& a;
  hipStream_t s;
  template <int G, int V>
  hipError_t operator()() const {
    // the kernel with sums in LDS has no registers to spare for it
    bwd_kernel<T, G, V, kEven, kJoin, kOdd && V == 1 && (G > 128)>
        <<<dim3(static_cast<unsigned>(a.parts)), dim3(bwd_threads<G>()), 0, s>>>(a);
    return hipGetLastError();
  }
};

template <class T, bool kJoin>
hipError_t reg_fwd(const NormFwdArgs& a, hipStream_t s) {
  return a.cols % 8 == 0 ? fwd_shape<sizeof(T)>(a.cols, LaunchFwd<T, true, kJoin>{a, s})
                         : fwd_shape<sizeof(T)>(a.cols, LaunchFwd<T, false, kJoin>{a, s});
}
inline bool bwd_join(const NormBwdArgs& a) {
  return a.x_bar == nullptr || a.res_bar != nullptr || a.h_bar != nullptr || a.drop.threshold != 0;
}

// Whether any row of an operand starts at an odd element (of 16 bits).
inline bool odd_rows(const void* p, int64_t stride, int32_t rows) {
  return p != nullptr && ((reinterpret_cast<uintptr_t>(p) & 2) != 0 || (rows > 1 && (stride & 1) != 0));
}

template <class T, bool kJoin>
hipError_t reg_bwd(const NormBwdArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (a.cols > 1024 &&
        (odd_rows(a.h, a.hs, a.rows) || odd_rows(a.y_bar, a.ybs, a.rows) || odd_rows(a.h_bar, a.hbs, a.rows)))
      return a.cols % 8 == 0 ? bwd_shape(a.cols, LaunchBwd<T, true, kJoin, true>{a, s})
                             : bwd_shape(a.cols, LaunchBwd<T, false, kJoin, true>{a, s});
  }
  return a.cols % 8 == 0 ? bwd_shape(a.cols, LaunchBwd<T, true, kJoin, false>{a, s})
                         : bwd_shape(a.cols, LaunchBwd<T, false, kJoin, false>{a, s});
}

// The plain layer norm has kernels of its own: nothing in their loops depends on what the
// caller left out.
template <class T>
hipError_t launch_fwd(const NormFwdArgs& a, hipStream_t s) {
  if (a.cols <= kRegCols) {
    const bool join = a.res != nullptr || a.h != nullptr || a.drop.threshold != 0;
    return join ? reg_fwd<T, true>(a, s) : reg_fwd<T, false>(a, s);
  }
  fwd_long_kernel<T><<<dim3(static_cast<unsigned>(std::min(a.rows, 2048))), dim3(kLong), 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.cols <= kRegCols) {
    return bwd_join(a) ? reg_bwd<T, true>(a, s) : reg_bwd<T, false>(a, s);
  }
  if (a.x_bar != nullptr || a.res_bar != nullptr) {
    bwd_long_kernel<T><<<dim3(static_cast<unsigned>(std::min(a.rows, 2048))), dim3(kLong), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.w_bar == nullptr && a.b_bar == nullptr) return hipSuccess;
  const int64_t vecs = (static_cast<int64_t>(a.cols) + 7) / 8;
  bwd_long_cols_kernel<T><<<dim3(static_cast<unsigned>((vecs + kThreads - 1) / kThreads),
                                static_cast<unsigned>(a.parts)),
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
