// Layer norm row kernels, f16 rows.
#include "layer_norm.hpp"

namespace etpc {
namespace norm {
ETPC_NORM_TYPE(F16, f16)
}  // namespace norm
}  // namespace etpc
