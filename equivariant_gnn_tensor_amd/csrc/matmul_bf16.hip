// Matrix products over bf16 operands (see matmul.hpp).
#include "matmul.hpp"

namespace etpc::mm {
hipError_t launch_bf16(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s) {
  return launch<Bf16>(a, form, shape, s);
}
}  // namespace etpc::mm
