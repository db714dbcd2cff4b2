// Layer norm launchers and the second stage of the column sums.
#include "layer_norm.hpp"

namespace etpc {
namespace {

// A workgroup sums 16 adjacent columns of `part`: 64 slices of the rows, each in order, then
// the slices in order.  16 columns are one 64-byte segment of a row of `part`.  More workgroups
// than kMaxGroups walk on (a launch holds less than 2^32 threads).
constexpr int kCols = 16, kSlices = 64;
constexpr int64_t kMaxGroups = int64_t{1} << 20;

__global__ __launch_bounds__(kCols* kSlices) void parts_reduce_kernel(const float* __restrict__ part, int parts,
                                                                      int cols, int64_t total,
                                                                      float* w_bar, float* b_bar) {
  __shared__ float lds[kSlices][kCols];
  const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kCols; first < total;
       first += static_cast<int64_t>(gridDim.x) * kCols) {
    const int64_t c = first + lane;
    lds[slice][lane] = c < total ? sum_slice<kSlices>(part + c, total, slice, parts) : 0.f;
    __syncthreads();
    if (slice == 0 && c < total) {
      float s = 0.f;
#pragma unroll 8
      for (int q = 0; q < kSlices; ++q) s += lds[q][lane];
      if (c < cols) {
        if (w_bar != nullptr) w_bar[c] = s;
      } else if (b_bar != nullptr) {
        b_bar[c - cols] = s;
      }
    }
    __syncthreads();
  }
}

// Workgroups of the backward pass, each of which leaves one row of partial sums.  By waves a
// CU: 8 for fp32 rows; 16-bit rows of the join carry half the bytes a wave and want 12
// (65408 x 1024 bf16: 142 us with 8, 131 with 12); 16-bit rows that leave a quarter of
// their threads idle want 16 (50000 x 577 bf16: 103 us with 8, 77 with 16).  Three rows a
// group at least, once there are 128 workgroups: fewer sums to add up afterwards (1000 x
// 1024 fp32: 15.2 us with one row, 10.0 with three).
struct CountParts {
  int32_t rows, cols;
  bool wide, join;   // 32-bit elements; the join
  template <int G, int V>
  int operator()() const {
    constexpr int threads = norm::bwd_threads<G>(), per = threads / G;
    const bool idle = G > 64 && 4 * ((static_cast<int64_t>(cols) + 7) / 8) <= 3 * G * V;
    const int waves = idle && !wide ? 16 : join && !wide ? 12 : 8;
    const int64_t most = G > 512 ? 256 : 256 * waves / (threads / 64);   // from 640 threads on, one a CU
    const int64_t units = (static_cast<int64_t>(rows) + per - 1) / per;
    return static_cast<int>(std::min(units, std::max<int64_t>(128, std::min((units + 2) / 3, most))));
  }
};

}  // namespace

int norm_parts_most(int32_t rows, int32_t cols) {
  if (cols > norm::kRegCols) return std::min(rows, 32);
  return norm::bwd_shape(cols, CountParts{rows, cols, false, true});
}

hipError_t launch_parts_reduce(const float* part, int parts, int cols, float* w_bar, float* b_bar, hipStream_t s) {
  const int64_t total = 2 * static_cast<int64_t>(cols);
  const unsigned groups = static_cast<unsigned>(std::min((total + kCols - 1) / kCols, kMaxGroups));
  parts_reduce_kernel<<<dim3(groups), dim3(kCols * kSlices), 0, s>>>(part, parts, cols, total, w_bar, b_bar);
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, hipStream_t s) {
  return dtype == ETPC_F32 ? norm::fwd_f32(a, s) : dtype == ETPC_BF16 ? norm::fwd_bf16(a, s) : norm::fwd_f16(a, s);
}

int norm_parts(const NormBwdArgs& a, int dtype) {
  if (a.cols > norm::kRegCols) return std::min(a.rows, 32);
  return norm::bwd_shape(a.cols, CountParts{a.rows, a.cols, dtype == ETPC_F32, norm::bwd_join(a)});
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, hipStream_t s) {
  return dtype == ETPC_F32 ? norm::bwd_f32(a, s) : dtype == ETPC_BF16 ? norm::bwd_bf16(a, s) : norm::bwd_f16(a, s);
}

}  // namespace etpc
