// Dropout from a counter-based generator, over rows and over irreps features.
//
// y = kept ? x * scale : 0.  The mask is a function of (seed, offset, row, column) alone: it
// is generated where it is used and never stored, and the gradient applies the same mask
// again (the map is diagonal, hence its own adjoint).  One generator call serves eight
// columns with 16 bits each, so a thread takes eight columns.
//
// Memory bound at the rate of a large copy: 65408 x 1024 bf16 in 47 us, 5.7 TB/s.  Sixteen bits
// a column are what makes it so: a call is twenty 32 x 32 -> 64 bit products, each of which
// takes four cycles of a lane, about as long for eight bf16 columns as their 32 bytes.
// p is rounded to a multiple of 2^-16 and the scale belongs to the rounded p.
#include <algorithm>

#include "nodewise.hpp"
#include "rows.hpp"

namespace etpc {
namespace {

constexpr int kThreads = 256;

// q = floor(a / d) for 0 <= a < 2^31 by a multiplication: RowMap's magic of the divisor d.
__device__ inline uint32_t div_by(uint32_t a, const RowMap& m) { return (__umulhi(a, m.magic) + a) >> m.shift; }

// More workgroups than this walk on (a launch holds less than 2^32 threads).
constexpr int64_t kMaxGroups = int64_t{1} << 22;

// Thread t of workgroup b takes vector b * 256 + t of the rows * vecs vectors.  The
// workgroup divides its first index once in 64 bits; the threads divide what is left over.
template <class T, bool kEven>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T* x, int64_t xs, T* y, int64_t ys, int64_t total,
                                                           int cols, RowMap vecs, DropArgs d) {
  const uint64_t offset = d.threshold != 0 ? drop_offset(d) : 0;
  for (uint64_t first = static_cast<uint64_t>(blockIdx.x) * kThreads; first + threadIdx.x < static_cast<uint64_t>(total);
       first += static_cast<uint64_t>(gridDim.x) * kThreads) {
    const uint64_t row0 = first / static_cast<uint32_t>(vecs.div);
    const uint32_t left = static_cast<uint32_t>(first - row0 * static_cast<uint32_t>(vecs.div)) + threadIdx.x;
    const uint32_t q = div_by(left, vecs);
    const uint32_t vec = left - q * static_cast<uint32_t>(vecs.div);
    const int64_t row = static_cast<int64_t>(row0 + q);
    float v[8];
    load<8, kEven>(x + row * xs, static_cast<int>(8 * vec), cols, v);
    if (d.threshold != 0) drop8(v, philox(vec, static_cast<uint32_t>(row), offset, d.seed), d.threshold, d.scale);
    store<8, kEven>(y + row * ys, static_cast<int>(8 * vec), cols, v);
  }
}

// A thread takes four channels of one block of one node, with all 2l+1 components: they share
// one mask, so a kept channel turns under a rotation as before.  Two threads make the same
// generator call and use half of it each: the mask serves every component, and four channels
// a thread leave the loads of a wave without gaps (60.3 us with eight a thread, 54.8 so, for
// 16384 nodes of 128x0e+128x1o+128x2e+128x3o).
template <int D, bool kEven>
__device__ inline void drop_block(const float* x, float* y, int mul, int c, uint32_t w0, uint32_t w1,
                                  const DropArgs& d) {
  float v[D][4];
#pragma unroll
  for (int m = 0; m < D; ++m) load<4, kEven>(x + m * mul, c, mul, v[m]);
  const bool keep[4] = {(w0 & 0xFFFFu) >= d.threshold, (w0 >> 16) >= d.threshold, (w1 & 0xFFFFu) >= d.threshold,
                        (w1 >> 16) >= d.threshold};
#pragma unroll
  for (int m = 0; m < D; ++m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[m][j] = keep[j] ? v[m][j] * d.scale : 0.f;
    store<4, kEven>(y + m * mul, c, mul, v[m]);
  }
}

template <bool kEven>
__global__ __launch_bounds__(kThreads) void irreps_dropout_kernel(const IrrepTable t, const float* x, float* y,
                                                                  int32_t rows, DropArgs d) {
  const IrrepBlock k = t.blk[blockIdx.y];
  const uint32_t quads = static_cast<uint32_t>(k.mul + 3) / 4;
  const uint64_t total = static_cast<uint64_t>(rows) * quads, offset = d.threshold != 0 ? drop_offset(d) : 0;
  for (uint64_t first = static_cast<uint64_t>(blockIdx.x) * kThreads; first + threadIdx.x < total;
       first += static_cast<uint64_t>(gridDim.x) * kThreads) {
    const uint64_t row0 = first / quads;
    const uint32_t left = static_cast<uint32_t>(first - row0 * quads) + threadIdx.x, node = left / quads;
    const uint32_t row = static_cast<uint32_t>(row0) + node, q = left - node * quads;
    uint32_t w0 = 0, w1 = 0;   // threshold 0 keeps everything, at scale 1
    if (d.threshold != 0) {
      const Philox r = philox(static_cast<uint32_t>(k.group) + q / 2, row, offset, d.seed);
      w0 = (q & 1) ? r.w[2] : r.w[0];
      w1 = (q & 1) ? r.w[3] : r.w[1];
    }
    const int64_t at = static_cast<int64_t>(row) * t.dim + k.off;
    const int c = static_cast<int>(4 * q);
    if (k.l == 0) drop_block<1, kEven>(x + at, y + at, k.mul, c, w0, w1, d);
    else if (k.l == 1) drop_block<3, kEven>(x + at, y + at, k.mul, c, w0, w1, d);
    else if (k.l == 2) drop_block<5, kEven>(x + at, y + at, k.mul, c, w0, w1, d);
    else drop_block<7, kEven>(x + at, y + at, k.mul, c, w0, w1, d);
  }
}

unsigned groups_of(int64_t threads) {
  return static_cast<unsigned>(std::min((threads + kThreads - 1) / kThreads, kMaxGroups));
}

template <class T>
hipError_t rows_of(const void* x, int64_t xs, void* y, int64_t ys, int32_t rows, int32_t cols, const DropArgs& d,
                   hipStream_t s) {
  const int32_t vecs = (cols + 7) / 8;
  const int64_t total = static_cast<int64_t>(rows) * vecs;
  const auto kernel = cols % 8 == 0 ? dropout_kernel<T, true> : dropout_kernel<T, false>;
  kernel<<<dim3(groups_of(total)), dim3(kThreads), 0, s>>>(static_cast<const T*>(x), xs, static_cast<T*>(y), ys, total,
                                                           cols, make_rowmap(0, 0, vecs), d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, int64_t xs, void* y, int64_t ys, int32_t rows, int32_t cols, int dtype,
                          const DropArgs& d, hipStream_t s) {
  if (dtype == ETPC_F32) return rows_of<float>(x, xs, y, ys, rows, cols, d, s);
  if (dtype == ETPC_BF16) return rows_of<Bf16>(x, xs, y, ys, rows, cols, d, s);
  return rows_of<F16>(x, xs, y, ys, rows, cols, d, s);
}

hipError_t launch_irreps_dropout(const IrrepTable& t, const float* x, float* y, int32_t rows, const DropArgs& d,
                                 hipStream_t s) {
  int32_t most = 0;
  bool even = true;
  for (int k = 0; k < t.n; ++k) {
    most = std::max(most, (t.blk[k].mul + 3) / 4);
    even = even && t.blk[k].mul % 4 == 0;
  }
  const int64_t total = static_cast<int64_t>(rows) * most;
  const auto kernel = even ? irreps_dropout_kernel<true> : irreps_dropout_kernel<false>;
  kernel<<<dim3(groups_of(total), static_cast<unsigned>(t.n)), dim3(kThreads), 0, s>>>(t, x, y, rows, d);
  return hipGetLastError();
}

}  // namespace etpc
