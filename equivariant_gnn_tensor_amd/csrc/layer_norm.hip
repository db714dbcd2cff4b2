// Layer norm launchers and the second stage of the column sums.
#include "layer_norm.hpp"

namespace etpc {
namespace {

// A workgroup sums 16 adjacent columns of `part`: 64 slices of the rows, each in order, then
// the slices in order.  16 columns are one 64-byte segment of a row of `part`.
constexpr int kCols = 16, kSlices = 64;

__global__ __launch_bounds__(kCols* kSlices) void parts_reduce_kernel(const float* __restrict__ part, int parts,
                                                                      int cols, int64_t total,
                                                                      float* w_bar, float* b_bar) {
  __shared__ float lds[kSlices][kCols];
  const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + lane;
  float s = 0.f;
  if (c < total) {
    int p = slice;
    for (; p + 7 * kSlices < parts; p += 8 * kSlices) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[static_cast<int64_t>(p + i * kSlices) * total + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; p < parts; p += kSlices) s += part[p * total + c];
  }
  lds[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || c >= total) return;
#pragma unroll 8
  for (int q = 1; q < kSlices; ++q) s += lds[q][lane];
  if (c < cols) {
    if (w_bar != nullptr) w_bar[c] = s;
  } else if (b_bar != nullptr) {
    b_bar[c - cols] = s;
  }
}

struct CountParts {
  int32_t rows;
  template <int G, int V>
  int operator()() const {
    constexpr int per = norm::threads_of<G>() / G;
    constexpr int most = G == 1024 ? 256 : 256 * 8 / (norm::threads_of<G>() / 64);
    return static_cast<int>(std::min<int64_t>((static_cast<int64_t>(rows) + per - 1) / per, most));
  }
};

}  // namespace

// Workgroups of the backward pass, each of which leaves one row of partial sums.
int norm_parts(int32_t rows, int32_t cols) {
  return cols > norm::kRegCols ? std::min(rows, 32) : norm::by_cols_bwd(cols, CountParts{rows});
}

hipError_t launch_parts_reduce(const float* part, int parts, int cols, float* w_bar, float* b_bar, hipStream_t s) {
  const int64_t total = 2 * static_cast<int64_t>(cols);
  parts_reduce_kernel<<<dim3(static_cast<unsigned>((total + kCols - 1) / kCols)), dim3(kCols * kSlices), 0, s>>>(
      part, parts, cols, total, w_bar, b_bar);
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, hipStream_t s) {
  return dtype == ETPC_F32 ? norm::fwd_f32(a, s) : dtype == ETPC_BF16 ? norm::fwd_bf16(a, s) : norm::fwd_f16(a, s);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, hipStream_t s) {
  return dtype == ETPC_F32 ? norm::bwd_f32(a, s) : dtype == ETPC_BF16 ? norm::bwd_bf16(a, s) : norm::bwd_f16(a, s);
}

}  // namespace etpc
