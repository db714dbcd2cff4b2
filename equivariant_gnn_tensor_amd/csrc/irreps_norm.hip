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
// Memory bound, like the layer norm of rows.  The grid's y axis is the block, so every wave
// works on segments of one length; a group of lanes owns a segment in registers.
#include <algorithm>

#include "nodewise.hpp"
#include "rows.hpp"

namespace etpc {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVecs = 8;                  // vectors of four numbers a lane holds
constexpr int kRegNumbers = 64 * 4 * kVecs;

// Lanes of a segment: a power of two up to the wave, by the number of four-vectors.
__device__ inline int lanes_of(int vecs) {
  int g = 4;
  while (g < vecs && g < 64) g *= 2;
  return g;
}

// The sum over aligned groups of g lanes (4..64), g uniform in the workgroup.
__device__ inline float sum_lanes(float v, int g) {
  v = lane_sum<4>(v);
  if (g >= 8) v += dpp_f<0x141>(v);
  if (g >= 16) v += dpp_f<0x140>(v);
  if (g >= 32) v = add_lane16(v);
  if (g >= 64) v = add_lane32(v);
  return v;
}

__device__ inline void load4(const float* __restrict__ p, int e, int n, float (&v)[4]) {
  if (e + 4 <= n) {
    __builtin_memcpy(v, p + e, 16);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = e + k < n ? p[e + k] : 0.f;
  }
}
__device__ inline void store4(float* __restrict__ p, int e, int n, const float (&v)[4]) {
  if (e + 4 <= n) {
    __builtin_memcpy(p + e, v, 16);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (e + k < n) p[e + k] = v[k];
  }
}

// The gains (biases) of four adjacent numbers of a segment, channel of number e = e mod C.
__device__ inline void channel4(const float* __restrict__ p, int e, int n, int mul, float missing, float (&v)[4]) {
  int c = e % mul;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = p != nullptr && e + k < n ? p[c] : missing;
    c = c + 1 == mul ? 0 : c + 1;
  }
}

__global__ __launch_bounds__(kThreads) void irreps_norm_fwd_kernel(const IrrepTable t, const float* x, const float* w,
                                                                   const float* b, float eps, float* y, float* stats,
                                                                   int32_t rows) {
  const IrrepBlock k = t.blk[blockIdx.y];
  const int n = (2 * k.l + 1) * k.mul, vecs = (n + 3) / 4;
  const int G = lanes_of(vecs), lane = threadIdx.x & (G - 1), per = kThreads / G;
  const float inv_n = 1.f / static_cast<float>(n);
  const float* gain = w != nullptr ? w + k.ch : nullptr;
  const float* bias = b != nullptr && k.bias >= 0 ? b + k.bias : nullptr;
  if (n > kRegNumbers) {   // longer segments are read once for each sum and once for y
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWaves + threadIdx.x / 64;
    for (int64_t row = wave; row < rows; row += static_cast<int64_t>(gridDim.x) * kWaves) {
      const float* xr = x + row * t.dim + k.off;
      float s = 0.f, mean = 0.f;
      if (k.l == 0) {
        for (int e = 4 * lane; e < n; e += 256) {
          float v[4];
          load4(xr, e, n, v);
          s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        mean = sum_lanes(s, 64) / static_cast<float>(n);   // exact for a constant row
        s = 0.f;
      }
      for (int e = 4 * lane; e < n; e += 256) {
        float v[4];
        load4(xr, e, n, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < n) s = fmaf(v[j] - mean, v[j] - mean, s);
      }
      const float rstd = 1.f / sqrtf(fmaf(sum_lanes(s, 64), inv_n, eps));
      if (lane == 0 && stats != nullptr) {
        stats[2 * (row * t.n + blockIdx.y)] = mean;
        stats[2 * (row * t.n + blockIdx.y) + 1] = rstd;
      }
      for (int e = 4 * lane; e < n; e += 256) {
        float v[4], g[4], c[4];
        load4(xr, e, n, v);
        channel4(gain, e, n, k.mul, 1.f, g);
        channel4(bias, e, n, k.mul, 0.f, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf((v[j] - mean) * rstd, g[j], c[j]);
        store4(y + row * t.dim + k.off, e, n, v);
      }
    }
    return;
  }
  float g[kVecs][4], c[kVecs][4];
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (i * G < vecs) {
      channel4(gain, 4 * (lane + i * G), n, k.mul, 1.f, g[i]);
      channel4(bias, 4 * (lane + i * G), n, k.mul, 0.f, c[i]);
    }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / G; row < rows;
       row += static_cast<int64_t>(gridDim.x) * per) {
    const float* xr = x + row * t.dim + k.off;
    float v[kVecs][4], s = 0.f, mean = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * G < vecs) load4(xr, 4 * (lane + i * G), n, v[i]);
    if (k.l == 0) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (i * G < vecs) s += (v[i][0] + v[i][1]) + (v[i][2] + v[i][3]);
      mean = sum_lanes(s, G) / static_cast<float>(n);
      s = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * G < vecs)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] -= mean;
          if (4 * (lane + i * G) + j < n) s = fmaf(v[i][j], v[i][j], s);
        }
    const float rstd = 1.f / sqrtf(fmaf(sum_lanes(s, G), inv_n, eps));
    if (lane == 0 && stats != nullptr) {
      stats[2 * (row * t.n + blockIdx.y)] = mean;
      stats[2 * (row * t.n + blockIdx.y) + 1] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * G < vecs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[i][j], c[i][j]);
        store4(y + row * t.dim + k.off, 4 * (lane + i * G), n, v[i]);
      }
  }
}

// Column sums stay in registers while a group walks its nodes; at the end each wave in turn
// adds its numbers to an LDS copy of the segment, and thread c sums the 2l+1 components of
// channel c: every order is fixed.
__global__ __launch_bounds__(kThreads) void irreps_norm_bwd_kernel(const IrrepTable t, const float* x,
                                                                   const float* y_bar, const float* stats,
                                                                   const float* w, float* x_bar, float* part,
                                                                   float* w_bar, float* b_bar, int32_t rows) {
  __shared__ float lds[2][kRegNumbers];
  const IrrepBlock k = t.blk[blockIdx.y];
  const int n = (2 * k.l + 1) * k.mul, vecs = (n + 3) / 4;
  const int G = lanes_of(vecs), lane = threadIdx.x & (G - 1), per = kThreads / G;
  const float inv_n = 1.f / static_cast<float>(n);
  const float* gain = w != nullptr ? w + k.ch : nullptr;
  const bool whole = gridDim.x == 1, sums = w_bar != nullptr || b_bar != nullptr;
  float* wo = whole ? w_bar : part + static_cast<int64_t>(blockIdx.x) * (t.channels + t.biases);
  float* bo = whole ? b_bar : wo + t.channels;
  if (n > kRegNumbers) {   // longer segments are read twice, and once more for the channel sums
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWaves + threadIdx.x / 64;
    for (int64_t row = wave; row < rows && x_bar != nullptr; row += static_cast<int64_t>(gridDim.x) * kWaves) {
      const float* xr = x + row * t.dim + k.off;
      const float* yr = y_bar + row * t.dim + k.off;
      const float mean = stats[2 * (row * t.n + blockIdx.y)], rstd = stats[2 * (row * t.n + blockIdx.y) + 1];
      float s0 = 0.f, s1 = 0.f;
      for (int e = 4 * lane; e < n; e += 256) {
        float v[4], d[4], g[4];
        load4(xr, e, n, v);
        load4(yr, e, n, d);
        channel4(gain, e, n, k.mul, 1.f, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s0 = fmaf(d[j], g[j], s0);
          s1 = fmaf(d[j] * g[j], (v[j] - mean) * rstd, s1);
        }
      }
      const float m0 = k.l == 0 ? sum_lanes(s0, 64) * inv_n : 0.f, m1 = sum_lanes(s1, 64) * inv_n;
      for (int e = 4 * lane; e < n; e += 256) {
        float v[4], d[4], g[4];
        load4(xr, e, n, v);
        load4(yr, e, n, d);
        channel4(gain, e, n, k.mul, 1.f, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = rstd * (fmaf(d[j], g[j], -m0) - (v[j] - mean) * rstd * m1);
        store4(x_bar + row * t.dim + k.off, e, n, v);
      }
    }
    if (!sums) return;
    for (int c = threadIdx.x; c < k.mul; c += kThreads) {
      float dw = 0.f, db = 0.f;
      for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float mean = stats[2 * (row * t.n + blockIdx.y)], rstd = stats[2 * (row * t.n + blockIdx.y) + 1];
        for (int e = c; e < n; e += k.mul) {
          const float d = y_bar[row * t.dim + k.off + e];
          dw = fmaf(d, (x[row * t.dim + k.off + e] - mean) * rstd, dw);
          db += d;
        }
      }
      if (wo != nullptr) wo[k.ch + c] = dw;
      if (bo != nullptr && k.bias >= 0) bo[k.bias + c] = db;
    }
    return;
  }
  float g[kVecs][4], dw[kVecs][4], db[kVecs][4];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (i * G < vecs) channel4(gain, 4 * (lane + i * G), n, k.mul, 1.f, g[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / G; row < rows;
       row += static_cast<int64_t>(gridDim.x) * per) {
    const float* xr = x + row * t.dim + k.off;
    const float* yr = y_bar + row * t.dim + k.off;
    float v[kVecs][4], d[kVecs][4], s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * G < vecs) {
        load4(xr, 4 * (lane + i * G), n, v[i]);
        load4(yr, 4 * (lane + i * G), n, d[i]);
      }
    const float mean = stats[2 * (row * t.n + blockIdx.y)], rstd = stats[2 * (row * t.n + blockIdx.y) + 1];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * G < vecs)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] = (v[i][j] - mean) * rstd;
          dw[i][j] = fmaf(d[i][j], v[i][j], dw[i][j]);
          db[i][j] += d[i][j];
          d[i][j] *= g[i][j];
          s0 += d[i][j];
          s1 = fmaf(d[i][j], v[i][j], s1);
        }
    if (x_bar == nullptr) continue;
    const float m0 = k.l == 0 ? sum_lanes(s0, G) * inv_n : 0.f, m1 = sum_lanes(s1, G) * inv_n;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * G < vecs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = rstd * (d[i][j] - fmaf(v[i][j], m1, m0));
        store4(x_bar + row * t.dim + k.off, 4 * (lane + i * G), n, v[i]);
      }
  }
  if (!sums) return;
  // the groups of a wave first: lane sums over equal positions
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (i * G < vecs)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        for (int o = G; o < 64; o *= 2) {
          dw[i][j] += __shfl_xor(dw[i][j], o);
          db[i][j] += __shfl_xor(db[i][j], o);
        }
  for (int q = 0; q < kWaves; ++q) {
    if (static_cast<int>(threadIdx.x / 64) == q && (threadIdx.x & 63) < static_cast<unsigned>(G)) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (i * G < vecs)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * (lane + i * G) + j;
            if (e < n) {
              lds[0][e] = q == 0 ? dw[i][j] : lds[0][e] + dw[i][j];
              lds[1][e] = q == 0 ? db[i][j] : lds[1][e] + db[i][j];
            }
          }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < k.mul; c += kThreads) {
    float sw = 0.f, sb = 0.f;
    for (int e = c; e < n; e += k.mul) {
      sw += lds[0][e];
      sb += lds[1][e];
    }
    if (wo != nullptr) wo[k.ch + c] = sw;
    if (bo != nullptr && k.bias >= 0) bo[k.bias + c] = sb;
  }
}

}  // namespace

// Four waves a workgroup, each at least one node; beyond 512 a block's waves fill the card.
int irreps_norm_parts(int32_t rows) { return std::min(rows / kWaves + (rows % kWaves != 0), 512); }

hipError_t launch_irreps_norm_fwd(const IrrepTable& t, const float* x, const float* w, const float* b, float eps,
                                  float* y, float* stats, int32_t rows, hipStream_t s) {
  const int groups = std::min(rows / kWaves + (rows % kWaves != 0), 2048);
  irreps_norm_fwd_kernel<<<dim3(static_cast<unsigned>(groups), static_cast<unsigned>(t.n)), dim3(kThreads), 0, s>>>(
      t, x, w, b, eps, y, stats, rows);
  return hipGetLastError();
}

hipError_t launch_irreps_norm_bwd(const IrrepTable& t, const float* x, const float* y_bar, const float* stats,
                                  const float* w, float* x_bar, float* w_bar, float* b_bar, float* part, int32_t rows,
                                  hipStream_t s) {
  irreps_norm_bwd_kernel<<<dim3(static_cast<unsigned>(irreps_norm_parts(rows)), static_cast<unsigned>(t.n)),
                           dim3(kThreads), 0, s>>>(t, x, y_bar, stats, w, x_bar, part, w_bar, b_bar, rows);
  return hipGetLastError();
}

}  // namespace etpc
