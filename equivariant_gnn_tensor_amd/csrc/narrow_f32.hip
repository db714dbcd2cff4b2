// The narrow dense layer over f32 rows (see narrow.hpp).
#include "narrow.hpp"

namespace etpc::narrow {
hipError_t fwd_f32(const FwdArgs& a, bool even, hipStream_t s) { return forward<float>(a, even, s); }
hipError_t bwd_f32(const BwdArgs& a, bool even, int groups, hipStream_t s) { return backward<float>(a, even, groups, s); }
}  // namespace etpc::narrow
