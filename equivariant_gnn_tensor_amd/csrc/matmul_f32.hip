// Matrix products over f32 operands (see matmul.hpp).
#include "matmul.hpp"

namespace etpc::mm {
hipError_t launch_f32(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s) {
  return launch<float>(a, form, shape, s);
}
}  // namespace etpc::mm
