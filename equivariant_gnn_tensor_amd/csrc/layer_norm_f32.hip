// Layer norm row kernels, f32 rows.
#include "layer_norm.hpp"

namespace etpc {
namespace norm {
ETPC_NORM_TYPE(float, f32)
}  // namespace norm
}  // namespace etpc
