// Gated join over f16 rows (see gated_join.hpp).
#include "gated_join.hpp"

namespace etpc::join {
hipError_t fwd_f16(const JoinFwdArgs& a, hipStream_t s) { return launch_fwd<F16>(a, s); }
hipError_t bwd_f16(const JoinBwdArgs& a, hipStream_t s) { return launch_bwd<F16>(a, s); }
}  // namespace etpc::join
