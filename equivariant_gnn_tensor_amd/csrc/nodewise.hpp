// Launchers of the node-wise operators: layer norm with its residual join, dropout, and
// the norm of irreps features (internal).
#pragma once

#include "common.hpp"
#include "philox.hpp"

namespace etpc {

// ---------------------------------------------------------------- layer norm over rows
// h = res + dropout(x) (res or dropout may be absent), y = (h - mean) rstd w + b.
// Row r of a matrix starts at pointer + r * stride elements.
struct NormFwdArgs {
  const void* x;
  const void* res;      // or null
  const float* w;       // or null: ones
  const float* b;       // or null: zeros
  void* y;
  void* h;              // or null
  float* mean;          // or null
  float* rstd;          // or null
  int64_t xs, ress, ys, hs;
  int32_t rows, cols;
  float eps;
  DropArgs drop;
};
hipError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, hipStream_t s);

// d = h_bar + (gradient of <y_bar, y> with respect to h); res_bar = d, x_bar = dropout(d),
// w_bar = sum_rows y_bar xhat, b_bar = sum_rows y_bar, the last two through `part`: `parts`
// rows of [2][cols] floats (none needed when that is 1).
struct NormBwdArgs {
  const void* h;
  const void* y_bar;
  const void* h_bar;    // or null: zeros
  const float* mean;
  const float* rstd;
  const float* w;       // or null: ones
  void* x_bar;          // or null
  void* res_bar;        // or null
  float* w_bar;         // or null
  float* b_bar;         // or null
  float* part;
  int64_t hs, ybs, hbs, xbs, rbs;
  int32_t rows, cols, parts;
  DropArgs drop;
};
// Workgroups of the backward pass for these arguments (not yet in a.parts), and the most that
// any element type and any of the optional operands give at this size.
int norm_parts(const NormBwdArgs& a, int dtype);
int norm_parts_most(int32_t rows, int32_t cols);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, hipStream_t s);

// w_bar[c], b_bar[c] = sum_{p < parts} part[p][0][c], part[p][1][c] in a fixed order; a null
// output is skipped.
hipError_t launch_parts_reduce(const float* part, int parts, int cols, float* w_bar, float* b_bar, hipStream_t s);

// ---------------------------------------------------------------- dropout over rows
hipError_t launch_dropout(const void* x, int64_t xs, void* y, int64_t ys, int32_t rows, int32_t cols, int dtype,
                          const DropArgs& d, hipStream_t s);

// ---------------------------------------------------------------- irreps features
constexpr int kMaxIrreps = 64;
// Block k of a feature row: [2l+1][mul] floats at off.  ch / bias: its first channel among
// the gains / biases (bias = -1: none).  group: its first group of eight channels.  wg, part:
// its first workgroup and its first partial sum in the irreps norm (irreps_deal).
struct IrrepBlock {
  int32_t off, mul, l, ch, bias, group, wg;
  int64_t part;
};
struct IrrepTable {
  int32_t n, dim, channels, biases, groups;
  IrrepBlock blk[kMaxIrreps];
};
hipError_t launch_irreps_dropout(const IrrepTable& t, const float* x, float* y, int32_t rows, const DropArgs& d,
                                 hipStream_t s);
// These fill in the table's deal of workgroups.
hipError_t launch_irreps_norm_fwd(IrrepTable& t, const float* x, const float* w, const float* b, float eps, float* y,
                                  float* stats, int32_t rows, hipStream_t s);
int64_t irreps_norm_part_floats(IrrepTable& t, int32_t rows);
hipError_t launch_irreps_norm_bwd(IrrepTable& t, const float* x, const float* y_bar, const float* stats,
                                  const float* w, float* x_bar, float* w_bar, float* b_bar, float* part, int32_t rows,
                                  hipStream_t s);

}  // namespace etpc
