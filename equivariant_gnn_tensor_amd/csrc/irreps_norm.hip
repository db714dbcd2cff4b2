// Layer norm of irreps features, forward and backward.
//
// A block of C channels of degree l is a segment of E = (2l+1) C adjacent numbers of a
// feature row.  With m = mean over the segment for l = 0 and m = 0 otherwise,
//   v = mean((x - m)^2),  r = 1 / sqrt(v + eps),  xh = (x - m) r,
//   y[c, mu] = w[c] xh[c, mu] + (0e only) b[c]
// and with g = y_bar w:
//   x_bar = r (g - (l = 0: mean(g)) - xh mean(g xh)),  w_bar[c] = sum_{node, mu} y_bar xh,
//   b_bar[c] = sum_node y_bar (0e).
// A rotation mixes the components mu of one channel only and leaves v unchanged, so the map
// commutes with it; a mean over channels may only be taken out, and a constant added, where
// the numbers are invariant.
//
// Memory bound: each operand is read once and each result written once.  A group of lanes
// owns a segment: lane j holds channels 4 j .. 4 j + 3 with all their components, so a
// gain, a bias and the gradients' sums are four registers a lane whatever the degree, and
// 64 channels fill 16 lanes exactly at every degree (against lanes that span the segment:
// backward of 65408 nodes of 64x0e+64x1o+64x2e 233 us -> 107).  That case reaches 91 us now,
// 5.0 TB/s, sums included; forward 60 us, 5.0 TB/s.  A large copy runs at 5.1 to 5.4.
#include <algorithm>

#include "nodewise.hpp"
#include "rows.hpp"

namespace etpc {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRegMul = 512;   // most channels a wave keeps in registers (two vectors a lane)

// Lanes of a segment: a power of two that covers its channels by fours, at most a wave.
__host__ __device__ inline int lanes_of(int mul) {
  int g = 1;
  while (4 * g < mul && g < 64) g *= 2;
  return g;
}

// Narrow blocks are read flat: lanes span the whole segment, four adjacent numbers each, and
// the components of a channel meet only in the gradients' sums at the end.  Channel by
// channel, lanes would read runs shorter than a cache line.  Below 24 channels backward
// (27542 nodes of 192x0e+8x2e+53x0e+32x1e+8x3o+6x1e 64 us -> 42; 36350 of 10x2o+48x3o+16x1e
// 62 -> 49, with 16 the bound 57), below 16 forward (25985 nodes of 88x0o+8x3o+8x1o+24x3o+
// 24x2o+88x0e 38 -> 34, 60000 of 16x0e+16x1o+16x2e 14.7, with 24 the bound 16.8).
constexpr int kFwdFlat = 16, kBwdFlat = 24;
__host__ __device__ inline bool is_flat(const IrrepBlock& b, int below) { return b.l == 0 || b.mul < below; }
// What the lanes of a group span: numbers of the segment, or channels.
__host__ __device__ inline int span_of(const IrrepBlock& b, int below) {
  return is_flat(b, below) ? (2 * b.l + 1) * b.mul : b.mul;
}

// The sums over aligned groups of g lanes, g uniform in the workgroup; two at once hide each
// other's latency.
template <int N>
__device__ inline void sum_lanes(float (&v)[N], int g) {
  const auto add = [&](auto step) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = step(v[i]);
  };
  if (g >= 2) add([](float x) { return x + dpp_f<0xB1>(x); });
  if (g >= 4) add([](float x) { return x + dpp_f<0x4E>(x); });
  if (g >= 8) add([](float x) { return x + dpp_f<0x141>(x); });
  if (g >= 16) add([](float x) { return x + dpp_f<0x140>(x); });
  if (g >= 32) add([](float x) { return add_lane16(x); });
  if (g >= 64) add([](float x) { return add_lane32(x); });
}
__device__ inline float sum_lanes(float v, int g) {
  float a[1] = {v};
  sum_lanes(a, g);
  return a[0];
}

// Where a lane's vector i lies among the channels of a component.  A vector that would start
// or end past the last channel is moved back to the last four: every access is one full
// vector inside the segment, and what it holds and writes there is bit for bit what the
// channels' owners hold and write.  Only sums tell the copies apart: element j counts from
// `skip` on.  Blocks of fewer than four channels (one lane each) go by elements.
template <int I, bool kEven>
struct Span {
  int mul, at[I], skip[I];
  __device__ inline Span(int lane, int lanes, int channels) : mul(channels) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = 4 * (lane + i * lanes);
      at[i] = tiny() ? 0 : min(c, mul - 4);
      skip[i] = tiny() ? 4 * min(i, 1) : min(c - at[i], 4);
    }
  }
  __device__ inline bool tiny() const { return !kEven && mul < 4; }
  __device__ inline bool counts(int i, int j) const {
    return kEven ? skip[i] == 0 : j >= skip[i] && j < mul;
  }
  // base is uniform, `offset` what the lane adds to it (floats)
  __device__ inline void load(const float* __restrict__ base, uint32_t offset, int i, float (&v)[4]) const {
    if (tiny()) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = j < mul ? base[offset + j] : 0.f;
    } else {
      __builtin_memcpy(v, base + (offset + static_cast<uint32_t>(at[i])), 16);
    }
  }
  __device__ inline void load_or(const float* __restrict__ base, int i, float missing, float (&v)[4]) const {
    if (base != nullptr) {
      load(base, 0, i, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = missing;
    }
  }
  __device__ inline void store(float* __restrict__ base, uint32_t offset, int i, const float (&v)[4]) const {
    if (tiny()) {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < mul) base[offset + j] = v[j];
    } else {
      __builtin_memcpy(base + (offset + static_cast<uint32_t>(at[i])), v, 16);
    }
  }
};

// A group's nodes: first + r step + group for the unrolled r.  Past the last node it reads
// the last one again (and writes nothing).
struct Node {
  int64_t base;      // uniform: the workgroup's first node of this step
  uint32_t offset;   // what the group adds to it
  bool live;
  __device__ inline Node(int64_t at, int group, int32_t rows) {
    base = at < rows ? at : rows - 1;
    const int64_t left = rows - 1 - base;
    live = at < rows && group <= left;
    offset = live ? group : static_cast<uint32_t>(left < group ? left : group);
  }
};

struct FwdArgs {
  const float* x;
  const float* w;
  const float* b;
  float* y;
  float* stats;
  float eps;
  int32_t rows;
};

struct BwdArgs {
  const float* x;
  const float* y_bar;
  const float* stats;
  const float* w;
  float* x_bar;
  float* w_bar;
  float* b_bar;
  float* part;
  int32_t rows;
  bool whole;   // one workgroup a block: sums go straight to w_bar and b_bar
};

// Which block a workgroup belongs to.
__device__ inline int block_of(const IrrepTable& t, int wg) {
  int k = 0;
  while (k + 1 < t.n && wg >= t.blk[k + 1].wg) ++k;
  return k;
}
__device__ inline int groups_of(const IrrepTable& t, int k) {
  return (k + 1 < t.n ? t.blk[k + 1].wg : t.groups) - t.blk[k].wg;
}

// The gains (or biases) of a lane's numbers: channel of number e of a flat segment = e mod C.
template <int D, int I, bool kEven>
__device__ inline void channel_values(const float* p, const Span<I, kEven>& span, const IrrepBlock& b, float missing,
                                      float (&v)[I][4]) {
#pragma unroll
  for (int i = 0; i < I; ++i) {
    if (D > 1 || b.l == 0) {
      span.load_or(p, i, missing, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[i][j] = p != nullptr && span.at[i] + j < span.mul ? p[(span.at[i] + j) % b.mul] : missing;
    }
  }
}

// D components of I vectors a lane (D = 1: a flat segment, of any degree), R nodes in flight a
// group.
template <int D, int I, int R, bool kEven>
__device__ inline void fwd_block(const IrrepTable& t, int k, int p, int parts, const FwdArgs& a) {
  const int mul = span_of(t.blk[k], kFwdFlat);
  const bool center = t.blk[k].l == 0;
  const int G = lanes_of(mul), lane = threadIdx.x & (G - 1), group = threadIdx.x / G, per = kThreads / G;
  const float inv_n = 1.f / static_cast<float>(D * mul);
  const Span<I, kEven> span(lane, G, mul);
  float w[I][4], b[I][4];
  channel_values<D>(a.w != nullptr ? a.w + t.blk[k].ch : nullptr, span, t.blk[k], 1.f, w);
  channel_values<D>(a.b != nullptr && t.blk[k].bias >= 0 ? a.b + t.blk[k].bias : nullptr, span, t.blk[k], 0.f, b);
  const int64_t step = static_cast<int64_t>(parts) * per;
  for (int64_t first = static_cast<int64_t>(p) * per; first < a.rows; first += R * step) {
    float v[R][D][I][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Node q(first + r * step, group, a.rows);
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < I; ++i)
          span.load(a.x + (q.base * t.dim + t.blk[k].off + d * mul), q.offset * t.dim, i, v[r][d][i]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Node q(first + r * step, group, a.rows);
      float s = 0.f, mean = 0.f, off = 0.f;
      if (D == 1 && center) {
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s += span.counts(i, j) ? v[r][0][i][j] : 0.f;
        mean = sum_lanes(s, G) / static_cast<float>(mul);   // one rounding, s * (1 / n) has two
        s = 0.f;
      }
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (D == 1) v[r][d][i][j] -= mean;
            const float c = span.counts(i, j) ? v[r][d][i][j] : 0.f;
            s = fmaf(c, c, s);
            if (D == 1) off += c;
          }
      if (D == 1 && center) {
        float both[2] = {s, off};
        sum_lanes(both, G);
        s = both[0];
        off = both[1] * inv_n;   // what the rounded mean is off by
      } else {
        s = sum_lanes(s, G);
        off = 0.f;
      }
      const float rstd = norm_rstd(s, off, inv_n, a.eps);
      if (!q.live) continue;
      if (a.stats != nullptr) {   // every lane of the group, the same bits
        float* st = a.stats + 2 * (q.base * t.n + k);
        st[2 * q.offset * t.n] = norm_mean(mean, off, rstd);
        st[2 * q.offset * t.n + 1] = rstd;
      }
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < I; ++i) {
          float o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = fmaf((v[r][d][i][j] - off) * rstd, w[i][j], b[i][j]);
          span.store(a.y + (q.base * t.dim + t.blk[k].off + d * mul), q.offset * t.dim, i, o);
        }
    }
  }
}

__device__ inline void load4_or(const float* __restrict__ p, int c, int n, float missing, float (&v)[4]) {
  if (p != nullptr) {
    load<4, false>(p, c, n, v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = missing;
  }
}

// Segments of more channels: a wave reads its segment once for each sum and once for y.
__device__ inline void fwd_long(const IrrepTable& t, int k, int p, int parts, const FwdArgs& a) {
  const int mul = t.blk[k].mul, n = (2 * t.blk[k].l + 1) * mul, lane = threadIdx.x & 63;
  const float inv_n = 1.f / static_cast<float>(n);
  const float* w = a.w != nullptr ? a.w + t.blk[k].ch : nullptr;
  const float* b = a.b != nullptr && t.blk[k].bias >= 0 ? a.b + t.blk[k].bias : nullptr;
  for (int64_t row = static_cast<int64_t>(p) * kWaves + threadIdx.x / 64; row < a.rows;
       row += static_cast<int64_t>(parts) * kWaves) {
    const float* x = a.x + row * t.dim + t.blk[k].off;
    float s = 0.f, mean = 0.f, off = 0.f;
    if (n == mul) {
      for (int e = 4 * lane; e < n; e += 256) {
        float v[4];
        load<4, false>(x, e, n, v);
        s += (v[0] + v[1]) + (v[2] + v[3]);
      }
      mean = sum_lanes(s, 64) / static_cast<float>(n);
      s = 0.f;
    }
    for (int e = 4 * lane; e < n; e += 256) {
      float v[4];
      load<4, false>(x, e, n, v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < n) {
          s = fmaf(v[j] - mean, v[j] - mean, s);
          off += v[j] - mean;
        }
    }
    off = n == mul ? sum_lanes(off, 64) * inv_n : 0.f;
    const float rstd = norm_rstd(sum_lanes(s, 64), off, inv_n, a.eps);
    if (lane == 0 && a.stats != nullptr) {
      a.stats[2 * (row * t.n + k)] = norm_mean(mean, off, rstd);
      a.stats[2 * (row * t.n + k) + 1] = rstd;
    }
    for (int d = 0; d * mul < n; ++d)
      for (int c = 4 * lane; c < mul; c += 256) {
        float v[4], g[4], h[4];
        load<4, false>(x + d * mul, c, mul, v);
        load4_or(w, c, mul, 1.f, g);
        load4_or(b, c, mul, 0.f, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(((v[j] - mean) - off) * rstd, g[j], h[j]);
        store<4, false>(a.y + row * t.dim + t.blk[k].off + d * mul, c, mul, v);
      }
  }
}

template <int I, bool kEven>
__global__ __launch_bounds__(kThreads) void irreps_norm_fwd_kernel(const IrrepTable t, const FwdArgs a) {
  const int k = block_of(t, blockIdx.x), p = blockIdx.x - t.blk[k].wg, parts = groups_of(t, k), l = t.blk[k].l;
  if (I == 2 && t.blk[k].mul > kRegMul) return fwd_long(t, k, p, parts, a);
  if (is_flat(t.blk[k], kFwdFlat)) fwd_block<1, I, 4, kEven>(t, k, p, parts, a);
  else if (l == 1) fwd_block<3, I, 2, kEven>(t, k, p, parts, a);
  else if (l == 2) fwd_block<5, I, 1, kEven>(t, k, p, parts, a);
  else fwd_block<7, I, 1, kEven>(t, k, p, parts, a);
}

// Where a workgroup of the backward pass leaves its sums: gains first, then biases.
__device__ inline void sum_outputs(const IrrepTable& t, int k, int p, const BwdArgs& a, float** wo, float** bo) {
  const IrrepBlock& q = t.blk[k];
  if (a.whole) {
    *wo = a.w_bar != nullptr ? a.w_bar + q.ch : nullptr;
    *bo = a.b_bar != nullptr && q.bias >= 0 ? a.b_bar + q.bias : nullptr;
  } else {
    *wo = a.part + q.part + static_cast<int64_t>(p) * (q.bias >= 0 ? 2 * q.mul : q.mul);
    *bo = q.bias >= 0 ? *wo + q.mul : nullptr;
  }
}

// A group keeps its channels' sums of y_bar xh and y_bar in registers while it walks its
// nodes; lanes, then waves are added at the end in a fixed order.
template <int D, int I, int R, bool kEven>
__device__ inline void bwd_block(const IrrepTable& t, int k, int p, int parts, const BwdArgs& a, float* lds) {
  const int mul = span_of(t.blk[k], kBwdFlat), channels = t.blk[k].mul;
  const bool center = t.blk[k].l == 0;
  const int G = lanes_of(mul), lane = threadIdx.x & (G - 1), group = threadIdx.x / G, per = kThreads / G;
  const float inv_n = 1.f / static_cast<float>(D * mul);
  const Span<I, kEven> span(lane, G, mul);
  float w[I][4], dw[I][4] = {}, db[I][4] = {};
  channel_values<D>(a.w != nullptr ? a.w + t.blk[k].ch : nullptr, span, t.blk[k], 1.f, w);
  const int64_t step = static_cast<int64_t>(parts) * per;
  for (int64_t first = static_cast<int64_t>(p) * per; first < a.rows; first += R * step) {
    float v[R][D][I][4], g[R][D][I][4], mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Node q(first + r * step, group, a.rows);
      const float* st = a.stats + 2 * (q.base * t.n + k);
      mean[r] = D == 1 && center ? st[2 * q.offset * t.n] : 0.f;
      rstd[r] = st[2 * q.offset * t.n + 1];
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int64_t base = q.base * t.dim + t.blk[k].off + d * mul;
          span.load(a.x + base, q.offset * t.dim, i, v[r][d][i]);
          span.load(a.y_bar + base, q.offset * t.dim, i, g[r][d][i]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Node q(first + r * step, group, a.rows);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& x = v[r][d][i][j];
            float& y = g[r][d][i][j];
            x = (D == 1 ? x - mean[r] : x) * rstd[r];
            if (q.live) {
              dw[i][j] = fmaf(y, x, dw[i][j]);
              if (D == 1) db[i][j] += y;
            }
            y *= w[i][j];
            const float c = span.counts(i, j) ? y : 0.f;
            if (D == 1) s0 += c;
            s1 = fmaf(c, x, s1);
          }
      if (a.x_bar == nullptr) continue;
      float m0 = 0.f, m1;
      if (D == 1 && center) {
        float both[2] = {s0, s1};
        sum_lanes(both, G);
        m0 = both[0] * inv_n;
        m1 = both[1] * inv_n;
      } else {
        m1 = sum_lanes(s1, G) * inv_n;
      }
      if (!q.live) continue;
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < I; ++i) {
          float o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = rstd[r] * (g[r][d][i][j] - fmaf(v[r][d][i][j], m1, m0));
          span.store(a.x_bar + (q.base * t.dim + t.blk[k].off + d * mul), q.offset * t.dim, i, o);
        }
    }
  }
  if (a.w_bar == nullptr && a.b_bar == nullptr) return;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      for (int o = G; o < 64; o *= 2) {
        dw[i][j] += __shfl_xor(dw[i][j], o);
        if (D == 1) db[i][j] += __shfl_xor(db[i][j], o);
      }
      const int wave = threadIdx.x / 64;
      if ((threadIdx.x & 63) < static_cast<unsigned>(G) && span.counts(i, j)) {
        const int c = span.at[i] + j;
        lds[wave * kRegMul + c] = dw[i][j];
        if (D == 1) lds[(kWaves + wave) * kRegMul + c] = db[i][j];
      }
    }
  __syncthreads();
  float *wo, *bo;
  sum_outputs(t, k, p, a, &wo, &bo);
  for (int c = threadIdx.x; c < channels; c += kThreads) {
    float sw = 0.f, sb = 0.f;
    for (int e = c; e < mul; e += channels)   // the components of a flat segment
#pragma unroll
      for (int q = 0; q < kWaves; ++q) sw += lds[q * kRegMul + e];
    if (wo != nullptr) wo[c] = sw;
    if (D == 1 && bo != nullptr) {
#pragma unroll
      for (int q = 0; q < kWaves; ++q) sb += lds[(kWaves + q) * kRegMul + c];
      bo[c] = sb;
    }
  }
}

__device__ inline void bwd_long(const IrrepTable& t, int k, int p, int parts, const BwdArgs& a) {
  const int mul = t.blk[k].mul, n = (2 * t.blk[k].l + 1) * mul, lane = threadIdx.x & 63;
  const float inv_n = 1.f / static_cast<float>(n);
  const float* w = a.w != nullptr ? a.w + t.blk[k].ch : nullptr;
  for (int64_t row = static_cast<int64_t>(p) * kWaves + threadIdx.x / 64; row < a.rows && a.x_bar != nullptr;
       row += static_cast<int64_t>(parts) * kWaves) {
    const int64_t at = row * t.dim + t.blk[k].off;
    const float mean = a.stats[2 * (row * t.n + k)], rstd = a.stats[2 * (row * t.n + k) + 1];
    float s0 = 0.f, s1 = 0.f;
    for (int d = 0; d * mul < n; ++d)
      for (int c = 4 * lane; c < mul; c += 256) {
        float v[4], y[4], g[4];
        load<4, false>(a.x + at + d * mul, c, mul, v);
        load<4, false>(a.y_bar + at + d * mul, c, mul, y);
        load4_or(w, c, mul, 1.f, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s0 = fmaf(y[j], g[j], s0);
          s1 = fmaf(y[j] * g[j], (v[j] - mean) * rstd, s1);
        }
      }
    const float m0 = n == mul ? sum_lanes(s0, 64) * inv_n : 0.f, m1 = sum_lanes(s1, 64) * inv_n;
    for (int d = 0; d * mul < n; ++d)
      for (int c = 4 * lane; c < mul; c += 256) {
        float v[4], y[4], g[4];
        load<4, false>(a.x + at + d * mul, c, mul, v);
        load<4, false>(a.y_bar + at + d * mul, c, mul, y);
        load4_or(w, c, mul, 1.f, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = rstd * (fmaf(y[j], g[j], -m0) - (v[j] - mean) * rstd * m1);
        store<4, false>(a.x_bar + at + d * mul, c, mul, v);
      }
  }
  if (a.w_bar == nullptr && a.b_bar == nullptr) return;
  float *wo, *bo;
  sum_outputs(t, k, p, a, &wo, &bo);
  for (int c = threadIdx.x; c < mul; c += kThreads) {
    float dw = 0.f, db = 0.f;
    for (int64_t row = p; row < a.rows; row += parts) {
      const int64_t at = row * t.dim + t.blk[k].off;
      const float mean = a.stats[2 * (row * t.n + k)], rstd = a.stats[2 * (row * t.n + k) + 1];
      for (int e = c; e < n; e += mul) {
        const float y = a.y_bar[at + e];
        dw = fmaf(y, (a.x[at + e] - mean) * rstd, dw);
        db += y;
      }
    }
    if (wo != nullptr) wo[c] = dw;
    if (bo != nullptr) bo[c] = db;
  }
}

template <int I, bool kEven>
__global__ __launch_bounds__(kThreads) void irreps_norm_bwd_kernel(const IrrepTable t, const BwdArgs a) {
  __shared__ float lds[2 * kWaves * kRegMul];
  const int k = block_of(t, blockIdx.x), p = blockIdx.x - t.blk[k].wg, parts = groups_of(t, k), l = t.blk[k].l;
  if (I == 2 && t.blk[k].mul > kRegMul) return bwd_long(t, k, p, parts, a);
  if (is_flat(t.blk[k], kBwdFlat)) bwd_block<1, I, 4, kEven>(t, k, p, parts, a, lds);
  else if (l == 1) bwd_block<3, I, 2, kEven>(t, k, p, parts, a, lds);
  else if (l == 2) bwd_block<5, I, 1, kEven>(t, k, p, parts, a, lds);
  else bwd_block<7, I, 1, kEven>(t, k, p, parts, a, lds);
}

// Second stage of the sums: a workgroup takes 16 adjacent columns of one block (gains, then
// biases), 64 slices of its rows of `part` in order each (eight loads in flight), then the
// slices in order.
constexpr int kCols = 16, kSlices = 64;

__global__ __launch_bounds__(kCols* kSlices) void irreps_parts_kernel(const IrrepTable t, const BwdArgs a) {
  __shared__ float lds[kSlices][kCols];
  const IrrepBlock& q = t.blk[blockIdx.y];
  const int width = q.bias >= 0 ? 2 * q.mul : q.mul, parts = groups_of(t, blockIdx.y);
  const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  const int c = blockIdx.x * kCols + lane;
  lds[slice][lane] = c < width ? sum_slice<kSlices>(a.part + q.part + c, width, slice, parts) : 0.f;
  __syncthreads();
  if (slice != 0 || c >= width) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < kSlices; ++i) s += lds[i][lane];
  if (c < q.mul) {
    if (a.w_bar != nullptr) a.w_bar[q.ch + c] = s;
  } else if (a.b_bar != nullptr) {
    a.b_bar[q.bias + c - q.mul] = s;
  }
}

// Blocks past 256 channels take two vectors a lane, and only channel counts that are no
// multiple of four need the code for ends inside a vector.
bool is_wide(const IrrepTable& t) {
  return std::any_of(t.blk, t.blk + t.n, [](const IrrepBlock& b) { return b.mul > 256; });
}
bool is_even(const IrrepTable& t, int below) {
  return std::all_of(t.blk, t.blk + t.n, [below](const IrrepBlock& b) { return span_of(b, below) % 4 == 0; });
}

}  // namespace

// Workgroups, resident all at once.  Fewer than fit measured best where a row is 4096 bytes
// (65408 nodes of 64x0e+64x1o+64x2e+64x3o: forward 116 us with 1024, 129 with 1536, 134 with
// 2048; backward 163 with 512, 168 with 768, 183 with 896, 179 with 1024); other rows differ
// by a few per cent between these.
constexpr int kFwdGroups = 1024, kBwdGroups = 768, kBwdGroupsWide = 512;

// Nodes a group has in flight.
int in_flight(const IrrepBlock& b, int below) { return is_flat(b, below) ? 4 : b.l == 1 ? 2 : 1; }

// Deals about `total` workgroups to the blocks so that all blocks walk the nodes at one pace:
// the rows in flight are one window of memory.  At least one workgroup each and no more than
// the nodes fill; single_step: one where a single step takes every node (the backward
// pass then often needs no second stage: 64 nodes of 8x0e+8x1o 7.8 us -> 5.3).  Lays out the
// rows of partial sums too; returns the floats these need.
int64_t irreps_deal(IrrepTable& t, int32_t rows, int total, int below, bool single_step) {
  double weight = 0.0;
  for (int k = 0; k < t.n; ++k)
    weight += static_cast<double>(lanes_of(span_of(t.blk[k], below))) / in_flight(t.blk[k], below);
  int64_t floats = 0;
  t.groups = 0;
  for (int k = 0; k < t.n; ++k) {
    IrrepBlock& q = t.blk[k];
    const int lanes = lanes_of(span_of(q, below)), per = kThreads / lanes;
    const bool one = single_step && static_cast<int64_t>(per) * in_flight(q, below) >= rows;
    const int64_t need = one ? 1 : (static_cast<int64_t>(rows) + per - 1) / per;
    const int64_t share = static_cast<int64_t>(total * lanes / (in_flight(q, below) * weight) + 0.5);
    const int64_t parts = std::max<int64_t>(1, std::min(need, share));
    q.wg = t.groups;
    q.part = floats;
    t.groups += static_cast<int32_t>(parts);
    floats += parts * (q.bias >= 0 ? 2 * q.mul : q.mul);
  }
  return t.groups > t.n ? floats : 0;
}

hipError_t launch_irreps_norm_fwd(IrrepTable& t, const float* x, const float* w, const float* b, float eps, float* y,
                                  float* stats, int32_t rows, hipStream_t s) {
  irreps_deal(t, rows, kFwdGroups, kFwdFlat, false);
  const FwdArgs a{x, w, b, y, stats, eps, rows};
  const bool even = is_even(t, kFwdFlat);
  const auto kernel = is_wide(t) ? (even ? irreps_norm_fwd_kernel<2, true> : irreps_norm_fwd_kernel<2, false>)
                                 : (even ? irreps_norm_fwd_kernel<1, true> : irreps_norm_fwd_kernel<1, false>);
  kernel<<<dim3(static_cast<unsigned>(t.groups)), dim3(kThreads), 0, s>>>(t, a);
  return hipGetLastError();
}

int64_t irreps_norm_part_floats(IrrepTable& t, int32_t rows) {
  return irreps_deal(t, rows, is_wide(t) ? kBwdGroupsWide : kBwdGroups, kBwdFlat, true);
}

hipError_t launch_irreps_norm_bwd(IrrepTable& t, const float* x, const float* y_bar, const float* stats,
                                  const float* w, float* x_bar, float* w_bar, float* b_bar, float* part, int32_t rows,
                                  hipStream_t s) {
  const bool whole = irreps_norm_part_floats(t, rows) == 0;
  const BwdArgs a{x, y_bar, stats, w, x_bar, w_bar, b_bar, part, rows, whole};
  const bool even = is_even(t, kBwdFlat);
  const auto kernel = is_wide(t) ? (even ? irreps_norm_bwd_kernel<2, true> : irreps_norm_bwd_kernel<2, false>)
                                 : (even ? irreps_norm_bwd_kernel<1, true> : irreps_norm_bwd_kernel<1, false>);
  kernel<<<dim3(static_cast<unsigned>(t.groups)), dim3(kThreads), 0, s>>>(t, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || whole || (w_bar == nullptr && b_bar == nullptr)) return e;
  int64_t most = 0;
  for (int k = 0; k < t.n; ++k) most = std::max<int64_t>(most, int64_t{t.blk[k].bias >= 0 ? 2 : 1} * t.blk[k].mul);
  irreps_parts_kernel<<<dim3(static_cast<unsigned>((most + kCols - 1) / kCols), static_cast<unsigned>(t.n)),
                        dim3(kCols * kSlices), 0, s>>>(t, a);
  return hipGetLastError();
}

}  // namespace etpc
