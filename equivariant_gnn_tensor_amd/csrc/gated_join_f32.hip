// Gated join over f32 rows (see gated_join.hpp).
#include "gated_join.hpp"

namespace etpc::join {
hipError_t fwd_f32(const JoinFwdArgs& a, hipStream_t s) { return launch_fwd<float>(a, s); }
hipError_t bwd_f32(const JoinBwdArgs& a, hipStream_t s) { return launch_bwd<float>(a, s); }
}  // namespace etpc::join
