// Launchers of the dense layer between narrow rows (internal).
#pragma once

#include "common.hpp"

namespace etpc {
namespace narrow {

// Strides in elements.  by_out: w[i ldw + o], else w[o ldw + i].
struct FwdArgs {
  const void* x;
  const void* w;
  const float* b;       // or null
  const void* res;      // or null
  void* y;
  void* z;              // or null
  int64_t xs, ldw, ress, ys, zs;
  int32_t rows, n_in, n_out, act;
  bool by_out;
};
struct BwdArgs {
  const void* x;        // read with w_sums
  const void* w;        // read with x_bar
  const void* y_bar;
  const void* z;        // or null: act is none
  void* x_bar;          // or null
  float* part;          // or null; [groups][n_in n_out + n_out], w_bar's part as [n_in][n_out] (wb_by_out) or [n_out][n_in]
  int64_t xs, ldw, ybs, zs, xbs;
  int32_t rows, n_in, n_out, act;
  bool by_out, wb_by_out, w_sums;   // w_sums: w_bar is wanted (its part is zeros otherwise)
};

constexpr int kMost = 128;
// The backward kernel keeps all of w_bar in a wave's registers, four tiles of 32 x 32, beside two rows'
// worth of y_bar and z.
inline bool fits_bwd(int64_t n_in, int64_t n_out) {
  const auto tiles = [](int64_t n) { return n <= 32 ? 1 : n <= 64 ? 2 : 4; };
  return n_in <= kMost && n_out <= kMost && tiles(n_out) <= 2 && tiles(n_in) * tiles(n_out) <= 4;
}
int bwd_groups(int64_t rows);
hipError_t run_fwd(const FwdArgs& a, int dtype, hipStream_t s);
hipError_t run_bwd(const BwdArgs& a, int dtype, hipStream_t s);

hipError_t fwd_f32(const FwdArgs& a, bool even, hipStream_t s);
hipError_t fwd_bf16(const FwdArgs& a, bool even, hipStream_t s);
hipError_t fwd_f16(const FwdArgs& a, bool even, hipStream_t s);
hipError_t bwd_f32(const BwdArgs& a, bool even, int groups, hipStream_t s);
hipError_t bwd_bf16(const BwdArgs& a, bool even, int groups, hipStream_t s);
hipError_t bwd_f16(const BwdArgs& a, bool even, int groups, hipStream_t s);

}  // namespace narrow
}  // namespace etpc
