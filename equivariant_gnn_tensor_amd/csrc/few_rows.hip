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
    constexpr unsigned cols = 8 * 16 / sizeof(T);
    few::across_kernel<T, M><<<groups(cols, 1 << 18), dim3(few::kAcrossThreads), 0, s>>>(a);
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
