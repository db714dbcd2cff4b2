// Launchers of the gated join and the second stage of its column sums.
#include "gated_join.hpp"

namespace etpc {
namespace {

// A workgroup sums 64 adjacent columns of `part`: 16 slices of the parts, each in order, then the
// slices in order (512 parts of 5 x 2047 sums: 6.3 us; 10.9 with 16 columns and 64 slices).
constexpr int kCols = 64, kSlices = 16;
struct Bars5 {
  float* out[5];
};
__global__ __launch_bounds__(kCols* kSlices) void parts_kernel(const float* __restrict__ part, int parts, int cols,
                                                               Bars5 bars) {
  __shared__ float lds[kSlices][kCols];
  const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  const int64_t total = 5 * static_cast<int64_t>(cols);
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kCols; first < total;
       first += static_cast<int64_t>(gridDim.x) * kCols) {
    const int64_t c = first + lane;
    lds[slice][lane] = c < total ? sum_slice<kSlices>(part + c, total, slice, parts) : 0.f;
    __syncthreads();
    if (slice == 0 && c < total) {
      float s = 0.f;
#pragma unroll 8
      for (int q = 0; q < kSlices; ++q) s += lds[q][lane];
#pragma unroll
      for (int j = 0; j < 5; ++j)
        if (c / cols == j && bars.out[j] != nullptr) bars.out[j][c - static_cast<int64_t>(j) * cols] = s;
    }
    __syncthreads();
  }
}

// Parts of the column sums: at least three rows' turns each, no more than are resident at once.  The call's
// time so, with twice as many and one turn, and with half as many: 4097 x 2047 fp32 59.7, 72.1, 55.3 us;
// 65408 x 1024 bf16 210, 246, 258.
struct BwdGroups {
  int32_t rows;
  template <int G>
  int operator()() const {
    constexpr int threads = join::bwd_threads<G>(), per = threads / G;
    const int64_t most = G > 512 ? 256 : 256 * 8 / (threads / 64);
    const int64_t units = (static_cast<int64_t>(rows) + per - 1) / per;
    return static_cast<int>(std::min(units, std::max<int64_t>(128, std::min((units + 2) / 3, most))));
  }
};

}  // namespace

bool join_means(int32_t cols) { return cols > join::kBwdCols; }

int join_parts(int32_t rows, int32_t cols) {
  return join_means(cols) ? std::min(rows, 32) : join::bwd_shape(cols, BwdGroups{rows});
}

hipError_t launch_join_fwd(const JoinFwdArgs& a, int dtype, hipStream_t s) {
  return dtype == ETPC_F32 ? join::fwd_f32(a, s) : dtype == ETPC_BF16 ? join::fwd_bf16(a, s) : join::fwd_f16(a, s);
}

hipError_t launch_join_bwd(const JoinBwdArgs& a, int dtype, hipStream_t s) {
  const hipError_t e =
      dtype == ETPC_F32 ? join::bwd_f32(a, s) : dtype == ETPC_BF16 ? join::bwd_bf16(a, s) : join::bwd_f16(a, s);
  if (e != hipSuccess || !a.sums || a.parts == 1) return e;
  const int64_t total = 5 * static_cast<int64_t>(a.cols);
  const unsigned groups = static_cast<unsigned>(std::min<int64_t>((total + kCols - 1) / kCols, 1 << 20));
  parts_kernel<<<dim3(groups), dim3(kCols * kSlices), 0, s>>>(a.part, a.parts, a.cols,
                                                             Bars5{{a.bar[0], a.bar[1], a.bar[2], a.bar[3], a.bar[4]}});
  return hipGetLastError();
}

}  // namespace etpc
