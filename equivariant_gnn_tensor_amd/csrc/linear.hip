// The dense layer beside its products: shapes of the products, the gradient through the
// activation with the bias's gradient, and sums of partial results.
#include <algorithm>

#include "activation.hpp"
#include "linear.hpp"
#include "narrow_args.hpp"
#include "rows.hpp"

namespace etpc {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGroups = int64_t{1} << 20;

// ---- z_bar = y_bar act'(z) and its column sums
// Memory bound: one pass, eight columns a thread, G threads along a row and 256 / G rows at a
// time.  A workgroup keeps its columns' sums in registers over all its rows and leaves one row
// of them; they are added up in a fixed order afterwards (65408 x 1024 f16 sums alone 30 us, 4.5 TB/s).
// z_bar is an operand of two products on the matrix cores, so it is rounded to the rows' type (2^-9 of
// itself in bf16); as two 16-bit numbers, like narrow rows have it, it would double their time (65408 x 1024 ->
// 4096 bf16 gelu: 920 of 1210 us).
struct SlopeShape {
  int g;        // threads along a row
  int groups;   // workgroups along a row
  int parts;
};
SlopeShape slope_shape(int32_t rows, int32_t cols) {
  const int vecs = cols / 8 + (cols % 8 != 0);
  SlopeShape s{8, 1, 1};
  while (s.g < kThreads && s.g < vecs) s.g *= 2;
  s.groups = (vecs + s.g - 1) / s.g;
  const int per = kThreads / s.g;
  const int64_t units = (static_cast<int64_t>(rows) + per - 1) / per;
  s.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((units + 3) / 4, 1024 / s.groups)));
  return s;
}

template <class T>
__global__ __launch_bounds__(kThreads) void slope_kernel(const SlopeArgs a, const SlopeShape sh) {
  __shared__ float lds[kThreads][8];
  const int part = blockIdx.x / sh.groups, group = blockIdx.x - part * sh.groups;
  const int lane = threadIdx.x & (sh.g - 1), row = threadIdx.x / sh.g, per = kThreads / sh.g;
  const int c = (group * sh.g + lane) * 8;
  float sum[8] = {};
  if (c < a.cols) {
    const int64_t step = static_cast<int64_t>(per) * sh.parts;
    for (int64_t r = static_cast<int64_t>(part) * per + row; r < a.rows; r += step) {
      float v[8], z[8];
      load<8, false>(static_cast<const T*>(a.y_bar) + r * a.ybs, c, a.cols, v);
      if (a.z != nullptr) {
        load<8, false>(static_cast<const T*>(a.z) + r * a.zs, c, a.cols, z);
        times_slope<sizeof(T) == 4>(v, z, a.act);
      }
      if (a.z_bar != nullptr) store<8, false>(static_cast<T*>(a.z_bar) + r * a.zbs, c, a.cols, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += c + k < a.cols ? v[k] : 0.f;
    }
  }
  if (a.part == nullptr) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) lds[threadIdx.x][k] = sum[k];
  __syncthreads();
  if (row == 0 && c < a.cols) {
    for (int i = 1; i < per; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += lds[i * sh.g + lane][k];
    store<8, false>(a.part + static_cast<int64_t>(part) * a.cols, c, a.cols, sum);
  }
}

// ---- sums of partial results
// kSlices threads share a number's parts: each takes every kSlices-th in order, then the slices
// in order.
template <class T, int kSlices>
__global__ __launch_bounds__(kThreads) void sum_parts_kernel(const float* __restrict__ part, int parts, int64_t rows,
                                                             int64_t cols, T* __restrict__ out, int64_t ld,
                                                             float* __restrict__ tail, int64_t tail_n) {
  constexpr int kNumbers = kThreads / kSlices;
  __shared__ float lds[kSlices][kNumbers];
  const int64_t total = rows * cols + tail_n;
  const int lane = threadIdx.x % kNumbers, slice = threadIdx.x / kNumbers;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kNumbers; first < total;
       first += static_cast<int64_t>(gridDim.x) * kNumbers) {
    const int64_t i = first + lane;
    float s = i < total ? sum_slice<kSlices>(part + i, total, slice, parts) : 0.f;
    if (kSlices > 1) {
      lds[slice][lane] = s;
      __syncthreads();
      if (slice == 0) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < kSlices; ++q) s += lds[q][lane];
      }
    }
    if (slice == 0 && i < total) {
      if (i >= rows * cols) {
        if (tail != nullptr) tail[i - rows * cols] = s;
      } else if (out != nullptr) {
        const int64_t r = i / cols;
        out[r * ld + (i - r * cols)] = static_cast<T>(s);
      }
    }
    if (kSlices > 1) __syncthreads();
  }
}

template <class T>
hipError_t sum_parts(const float* part, int parts, int64_t rows, int64_t cols, void* out, int64_t ld, float* tail,
                     int64_t tail_n, hipStream_t s) {
  const int64_t total = rows * cols + tail_n;
  if (total == 0) return hipSuccess;
  const int slices = parts >= 16 ? 16 : 1, numbers = kThreads / slices;
  const dim3 grid(static_cast<unsigned>(std::min((total + numbers - 1) / numbers, kMaxGroups)));
  if (slices == 16)
    sum_parts_kernel<T, 16><<<grid, kThreads, 0, s>>>(part, parts, rows, cols, static_cast<T*>(out), ld, tail,
                                                        tail_n);
  else
    sum_parts_kernel<T, 1><<<grid, kThreads, 0, s>>>(part, parts, rows, cols, static_cast<T*>(out), ld, tail,
                                                        tail_n);
  return hipGetLastError();
}

// ---- the layer's epilogue over partial sums: four columns a thread
template <class T>
__global__ __launch_bounds__(kThreads) void layer_parts_kernel(const MatmulArgs a) {
  const int64_t per = (a.N + 3) / 4, total = per * a.M, size = static_cast<int64_t>(a.M) * a.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t m = i / per;
    const int n = static_cast<int>(i - m * per) * 4;
    float v[4] = {}, w[4];
    int p = 0;
    for (; p + 4 <= a.splits; p += 4) {   // four loads on their way
      float u[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) load<4, false>(a.part + (p + j) * size + m * a.N, n, a.N, u[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += u[j][k];
    }
    for (; p < a.splits; ++p) {
      load<4, false>(a.part + p * size + m * a.N, n, a.N, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += w[k];
    }
    if (a.bias != nullptr) {
      load<4, false>(a.bias, n, a.N, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += w[k];
    }
    if (a.z != nullptr) store<4, false>(static_cast<T*>(a.z) + m * a.ldz, n, a.N, v);
    if (a.act != ETPC_ACT_NONE) activate<sizeof(T) == 4>(v, a.act);
    if (a.res != nullptr) {
      load<4, false>(static_cast<const T*>(a.res) + m * a.ldres, n, a.N, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += w[k];
    }
    store<4, false>(static_cast<T*>(a.c) + m * a.ldc, n, a.N, v);
  }
}

// Bytes a lane with which an operand can go straight into LDS (0: it cannot): whole aligned pieces,
// offsets inside a tile in 31 bits.  n: its other index; cols: contiguous along that one.
int grain_of(const void* p, int64_t ld, int64_t n, int64_t k, bool cols, int64_t size) {
  const int64_t row = cols ? n : k;
  if (ld < row || 256 * ld * size >= 0x70000000) return 0;
  for (const int g : {16, 4})
    if (reinterpret_cast<uintptr_t>(p) % g == 0 && ld * size % g == 0 && row * size % g == 0) return g;
  return 0;
}

}  // namespace

int slope_parts(int32_t rows, int32_t cols) { return slope_shape(rows, cols).parts; }

hipError_t launch_slope(const SlopeArgs& a, int dtype, hipStream_t s) {
  const SlopeShape sh = slope_shape(a.rows, a.cols);
  const dim3 grid(static_cast<unsigned>(sh.parts) * static_cast<unsigned>(sh.groups));
  if (dtype == ETPC_F32)
    slope_kernel<float><<<grid, kThreads, 0, s>>>(a, sh);
  else if (dtype == ETPC_BF16)
    slope_kernel<Bf16><<<grid, kThreads, 0, s>>>(a, sh);
  else
    slope_kernel<F16><<<grid, kThreads, 0, s>>>(a, sh);
  return hipGetLastError();
}

hipError_t launch_sum_parts(const float* part, int parts, int64_t rows, int64_t cols, void* out, int64_t ld, float* tail,
                            int64_t tail_n, int dtype, hipStream_t s) {
  return dtype == ETPC_F32    ? sum_parts<float>(part, parts, rows, cols, out, ld, tail, tail_n, s)
         : dtype == ETPC_BF16 ? sum_parts<Bf16>(part, parts, rows, cols, out, ld, tail, tail_n, s)
                              : sum_parts<F16>(part, parts, rows, cols, out, ld, tail, tail_n, s);
}

hipError_t launch_layer_parts(const MatmulArgs& a, int dtype, hipStream_t s) {
  const int64_t units = ((a.N + 3) / 4 * static_cast<int64_t>(a.M) + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(std::min(units, kMaxGroups)));
  if (dtype == ETPC_F32)
    layer_parts_kernel<float><<<grid, kThreads, 0, s>>>(a);
  else if (dtype == ETPC_BF16)
    layer_parts_kernel<Bf16><<<grid, kThreads, 0, s>>>(a);
  else
    layer_parts_kernel<F16><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

// ---- narrow rows: whole chunks for every row of every operand?
namespace narrow {
namespace {
bool whole(const void* p, int64_t stride, int64_t n, int64_t size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0 && n * size % 16 == 0);
}
}  // namespace

int bwd_groups(int64_t rows) { return static_cast<int>(std::min<int64_t>((rows + 255) / 256, 256)); }

hipError_t run_fwd(const FwdArgs& a, int dtype, hipStream_t s) {
  const bool even = whole(a.x, a.xs, a.n_in, dtype == ETPC_F32 ? 4 : 2);
  return dtype == ETPC_F32 ? fwd_f32(a, even, s) : dtype == ETPC_BF16 ? fwd_bf16(a, even, s) : fwd_f16(a, even, s);
}

hipError_t run_bwd(const BwdArgs& a, int dtype, hipStream_t s) {
  const int64_t size = dtype == ETPC_F32 ? 4 : 2;
  const bool even = whole(a.part != nullptr ? a.x : nullptr, a.xs, a.n_in, size) && whole(a.y_bar, a.ybs, a.n_out, size) &&
                    whole(a.z, a.zs, a.n_out, size);
  const int groups = bwd_groups(a.rows);
  return dtype == ETPC_F32 ? bwd_f32(a, even, groups, s) : dtype == ETPC_BF16 ? bwd_bf16(a, even, groups, s) : bwd_f16(a, even, groups, s);
}
}  // namespace narrow

MatmulShape matmul_shape(const MatmulArgs& a, MatmulForm form, int dtype, bool sums) {
  const int64_t size = dtype == ETPC_F32 ? 4 : 2;
  MatmulShape s{64, 0, 1, a.K, 2};
  s.grain = std::min(grain_of(a.a, a.lda, a.M, a.K, form == MatmulForm::kColsCols, size),
                     grain_of(a.b, a.ldb, a.N, a.K, form != MatmulForm::kRowsRows, size));
  const auto tiles = [&](int64_t side) { return ((a.M + side - 1) / side) * ((a.N + side - 1) / side); };
  const int64_t bk = 128 / size, slices = (a.K + bk - 1) / bk;
  const int64_t narrow = std::min(a.M, a.N);
  int64_t splits = 1;
  if (sums) {
    // One round of the largest tile, two of the others, each workgroup at least 512 rows; where that leaves CUs
    // without work, the next smaller tile (16384 x 512 -> 512 bf16 37.0 us; 41.2 with the largest), and with
    // the smallest down to 128 rows (1000 x 776 -> 336 fp32 18.6 us; 69.0 with 128 x 128 and 512 rows).
    const auto ranges = [&](int64_t side, int64_t least) {
      return std::min(std::max<int64_t>(1, (side == 256 ? 256 : 512) / tiles(side)), std::max<int64_t>(1, a.K / least));
    };
    s.tile = 64;
    if (size == 2 && narrow >= 256 && tiles(256) * ranges(256, 512) >= 192) s.tile = 256;
    else if (narrow > 64 && tiles(128) * ranges(128, 512) >= 192) s.tile = 128;
    splits = ranges(s.tile, s.tile == 64 ? 128 : 512);
  } else {
    // The largest tile that leaves no CU idle.  bf16: 16384 x 1024 -> 1024 (256 tiles of 256 x 256) 39.5 us
    // and 44.3 with 128 x 128; 8192 x 1024 -> 1024 (128 of them) 31.8 and 22.9; 2048 x 1024 -> 2048 (256 of
    // 128 x 128) 15.3 and 18.2 with 64 x 64; 4096 x 2048 -> 512 (128) 26.0 and 20.0.  None that a narrow
    // C would leave half empty (65536 x 512 -> 64 15.1 and 22.7 with 256 x 256, fp32 43.4 and 76.8 with 128 x 128).
    s.tile = size == 2 && narrow > 128 && tiles(256) >= 256 ? 256 : narrow > 64 && tiles(128) >= 256 ? 128 : 64;
    // Few tiles and a long k: a tile's products take longer than the second launch that adds ranges of k
    // (a slice takes a CU about 0.45 us in fp32, 0.3 in 16 bits; 256 x 4096 -> 256 fp32 24.6 us, 78.6
    // whole; bf16 15.2 and 25.6).
    if (a.M > kFewRows && tiles(64) <= 128 && slices >= (size == 4 ? 12 : 20)) splits = std::min(512 / tiles(64), slices / 4);
  }
  const int64_t each = (slices + splits - 1) / splits * bk;
  s.k_split = static_cast<int>(std::min<int64_t>(each, a.K));
  s.splits = static_cast<int>((a.K + each - 1) / each);
  if (s.tile == 256 && s.grain != 16) s.tile = 128;
  // A third slice where every CU has all its 64 x 64 tiles at once, three at most, and waits for loads
  // (2048 x 4096 -> 768 bf16 31.3 us; 36.3 with two); fp32 waits for its products (4096 x 2048 -> 512 80
  // us with either).
  s.stages = s.tile == 64 && s.grain == 16 && size == 2 && tiles(64) * s.splits <= 768 ? 3 : 2;
  return s;
}

hipError_t launch_matmul(const MatmulArgs& args, MatmulForm form, int dtype, const MatmulShape& shape, hipStream_t s) {
  if (args.M <= kFewRows && form != MatmulForm::kColsCols && args.part == nullptr)
    return launch_few_rows(args, form == MatmulForm::kRowsRows, dtype, s);
  MatmulArgs a = args;
  a.splits = shape.splits;
  a.k_split = shape.k_split;
  return dtype == ETPC_F32    ? mm::launch_f32(a, form, shape, s)
         : dtype == ETPC_BF16 ? mm::launch_bf16(a, form, shape, s)
                              : mm::launch_f16(a, form, shape, s);
}

}  // namespace etpc
