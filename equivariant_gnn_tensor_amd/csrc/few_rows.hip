// Launches of the dense layer for one or two rows.
#include <algorithm>

#include "few_rows.hpp"

namespace etpc {
namespace {

template <class T, int M>
hipError_t launch(const MatmulArgs& a, bool along, hipStream_t s) {
  const auto groups = [&](unsigned outputs, unsigned most) { return dim3(std::min((a.N + outputs - 1) / outputs, most)); };
  if (along) {
    // one output a wave until there are enough waves for every CU
    if (a.N <= 4096)
      few::along_kernel<T, M, 1><<<groups(4, 1 << 20), dim3(few::kAlongThreads), 0, s>>>(a);
    else
      few::along_kernel<T, M, 4><<<groups(16, 1 << 20), dim3(few::kAlongThreads), 0, s>>>(a);
  } else {
    // 64 bytes of n a workgroup up to 64 workgroups of 128 bytes: 1 x 2047 -> 511 fp32 7.5 us (12.0 with 128),
    // 1 x 1024 -> 1024 5.5 (6.2), 1 x 4096 -> 4096 bf16 19.9 (26.2); past them 1 x 4096 -> 4096 fp32 24.6 (22.7),
    // 1 x 1024 -> 8192 15.5 (9.5).  Weights from memory each time.
    constexpr unsigned cols = 16 / sizeof(T);
    if (a.N <= 64 * 8 * static_cast<int>(cols))
      few::across_kernel<T, M, 4><<<groups(4 * cols, 1 << 18), dim3(few::kAcrossThreads), 0, s>>>(a);
    else
      few::across_kernel<T, M, 8><<<groups(8 * cols, 1 << 18), dim3(few::kAcrossThreads), 0, s>>>(a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch(const MatmulArgs& a, bool along, hipStream_t s) {
  static_assert(kFewRows == 2, "the rows below");
  return a.M == 1 ? launch<T, 1>(a, along, s) : launch<T, 2>(a, along, s);
}

}  // namespace

hipError_t launch_few_rows(const MatmulArgs& a, bool along, int dtype, hipStream_t s) {
  return dtype == ETPC_F32    ? launch<float>(a, along, s)
         : dtype == ETPC_BF16 ? launch<Bf16>(a, along, s)
                              : launch<F16>(a, along, s);
}

}  // namespace etpc
