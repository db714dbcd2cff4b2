// The narrow dense layer over f16 rows (see narrow.hpp).
#include "narrow.hpp"

namespace etpc::narrow {
hipError_t fwd_f16(const FwdArgs& a, bool even, hipStream_t s) { return forward<F16>(a, even, s); }
hipError_t bwd_f16(const BwdArgs& a, bool even, int groups, hipStream_t s) { return backward<F16>(a, even, groups, s); }
}  // namespace etpc::narrow
