// Layer norm row kernels, bf16 rows.
#include "layer_norm.hpp"

namespace etpc {
namespace norm {
ETPC_NORM_TYPE(Bf16, bf16)
}  // namespace norm
}  // namespace etpc
