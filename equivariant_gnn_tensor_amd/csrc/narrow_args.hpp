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
// Forward: a wave that works on 32 rows alone needs many of them, or little work on each, against the tiles
// of matmul.hpp.  Up to two tiles of 32 x 32 always (64 -> 32 silu: 3000 rows or less alike, 214980 bf16 13.6 us
// and 20.5 with the tiles, fp32 26.1 and 39.0).  With more, rows past what those tiles take in one round (65536
// in tiles of 128, 81920 in tiles of 64, some more where both load whole pieces; us here and with the tiles):
//   16 bits, n_out <= 64: 64 -> 64 65000 rows 11.2 and 9.1, 83000 12.7 and 10.7, 90000 12.7 and 12.9, 214980 20.7
//     and 22.7, 500000 36.2 and 47.9 (short of a round's end the tiles are ahead: 163000 18.0 and 16.1);
//     90 -> 50 83000 rows 17.8 and 16.0, 100000 20.9 and 26.4;
//   16 bits, n_out > 64: 33 -> 65 70000 rows 20.9 and 42.3; whole 16-byte pieces on both sides keep the tiles
//     (32 -> 128 100000 rows 21.4 and 18.6);
//   fp32, n_in <= 32: 32 -> 128 72000 rows 34.4 and 48.3, 60000 24.6 and 29.2, 40000 21.4 and 18.8;
//   fp32, four tiles: rows whose outputs end inside 64 bytes, which the tiles write in pieces (62 -> 62 100000 rows
//     33.3 and 56.3; 60 -> 60 83000 25.2 and 38.4, 70000 24.7 and 28.8; from 33 to 40 outputs alike within 40 %
//     either way), not others (64 -> 64 150000 rows 33.6 and 29.3; 48 -> 64 100000 26.0 and 27.6, 400000 75.5 and 70.5);
//   fp32, n_in > 64: whole pieces of x (96 -> 32 100000 rows 24.2 and 31.0; 75 -> 20 36.3 and 37.0, 150000 45.0
//     and 38.5), not with more than 32 outputs (127 -> 63 150000 rows 82.9 and 74.4);
//   fp32, eight tiles with n_out > 64: from 73 outputs on that end inside 64 bytes (50 -> 75 83000 rows 52.8 and
//     64.5; 50 -> 70 100000 67.6 and 54.2, 50 -> 80 60.2 and 42.9).
inline bool fits_fwd(int64_t rows, int64_t n_in, int64_t n_out, int32_t dtype) {
  if (n_in > kMost || n_out > kMost) return false;
  const int64_t size = dtype == ETPC_F32 ? 4 : 2;
  const bool aligned = n_in * size % 16 == 0 && n_out * size % 16 == 0;
  const int tiles = tiles_of(n_in) * tiles_of(n_out);
  if (tiles <= 2) return true;
  if (tiles > 8 || (tiles > 4 && aligned)) return false;
  if (rows <= (n_out > 64 ? 65536 : n_in > 64 || (size == 2 && aligned) ? 90000 : 81920)) return false;
  if (dtype != ETPC_F32) return n_out <= 64 || !aligned;
  if (n_in > 64) return n_out <= 32 && n_in % 4 == 0;
  if (n_out > 64) return n_in <= 32 || (n_out > 72 && n_out % 16 != 0);
  return n_out % 16 != 0;
}
// Backward: the kernel keeps all of w_bar in a wave's registers, four tiles of 32 x 32, beside two rows'
// worth of y_bar and z.  Four of them in fp32 take a wave longer than few rows are worth (64 -> 64: 20000 rows
// 33.8 us and 30.5 with the products apart, 50000 36.9 and 39.5; bf16 20.8 and 24.3, 22.8 and 30.2).
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
