// Gated join over bf16 rows (see gated_join.hpp).
#include "gated_join.hpp"

namespace etpc::join {
hipError_t fwd_bf16(const JoinFwdArgs& a, hipStream_t s) { return launch_fwd<Bf16>(a, s); }
hipError_t bwd_bf16(const JoinBwdArgs& a, hipStream_t s) { return launch_bwd<Bf16>(a, s); }
}  // namespace etpc::join
