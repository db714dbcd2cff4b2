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
inline int tiles_of(int64_t n) { return n <= 32 ? 1 : n <= 64 ? 2 : 4; }
// Forward: a wave that works on 32 rows alone needs many of them, or little work on each, against the tiles of
// matmul.hpp (us here and there, silu).  64 -> 32: 3000 rows or less alike, 214980 bf16 14.4 and 20.3, fp32
// 26.5 and 38.3; 64 -> 64 bf16: 65000 rows 10.8 and 9.0, 214980 22.6 and 23.8; 128 -> 32: 20.3 and 24.1,
// fp32 41.4 and 52.9; 63 -> 63: fp32 59.6 and 121.9, 3000 rows 13.1 and 8.5.  Beyond four tiles of 32 x 32 only
// where the tiles' loads are not aligned: 128 -> 64 bf16 32.5 and 27.5, 100 -> 60 37.3 and 47.1, 60 -> 100
// fp32 100.7 and 145.6; 128 -> 128 bf16 61.0 and 37.3.
inline bool fits_fwd(int64_t rows, int64_t n_in, int64_t n_out, int32_t dtype) {
  if (n_in > kMost || n_out > kMost) return false;
  const int64_t size = dtype == ETPC_F32 ? 4 : 2;
  const bool aligned = n_in * size % 16 == 0 && n_out * size % 16 == 0;
  const int tiles = tiles_of(n_in) * tiles_of(n_out);
  return tiles <= 2 || (rows > 65536 && tiles <= (aligned ? 4 : 8));
}
// Backward: the kernel keeps all of w_bar in a wave's registers, four tiles of 32 x 32, beside two rows'
// worth of y_bar and z.  Four of them in fp32 take a wave longer than few rows are worth (64 -> 64: 20000 rows
// 33.8 us and 30.5 with the products apart, 50000 37.3 and 39.5; bf16 20.2 and 24.3, 22.6 and 30.2).
inline bool fits_bwd(int64_t rows, int64_t n_in, int64_t n_out, int32_t dtype) {
  if (n_in > kMost || n_out > 64) return false;
  const int tiles = tiles_of(n_in) * tiles_of(n_out);
  return tiles <= 2 || (tiles <= 4 && (dtype != ETPC_F32 || rows > 32768));
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
