// The narrow dense layer over bf16 rows (see narrow.hpp).
#include "narrow.hpp"

namespace etpc::narrow {
hipError_t fwd_bf16(const FwdArgs& a, bool even, hipStream_t s) { return forward<Bf16>(a, even, s); }
hipError_t bwd_bf16(const BwdArgs& a, bool even, int groups, hipStream_t s) { return backward<Bf16>(a, even, groups, s); }
}  // namespace etpc::narrow
