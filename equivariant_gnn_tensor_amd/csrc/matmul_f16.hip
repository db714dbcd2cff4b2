// Matrix products over f16 operands (see matmul.hpp).
#include "matmul.hpp"

namespace etpc::mm {
hipError_t launch_f16(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s) {
  return launch<F16>(a, form, shape, s);
}
}  // namespace etpc::mm
