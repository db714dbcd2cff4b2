// Launchers of the gated residual join between two norms (internal).
#pragma once

#include "common.hpp"

namespace etpc {

// Row r of a matrix starts at pointer + r * stride elements; stats are [rows][4] floats:
// mean and rstd of x, mean and rstd of h.
struct JoinFwdArgs {
  const void* x;
  const void* gate;     // or null: open
  const void* res;      // or null: zeros
  const float* w1;      // or null: ones, zeros
  const float* b1;
  const float* scale;
  const float* w2;
  const float* b2;
  void* y;
  void* h;              // or null
  float* stats;         // or null
  int64_t xs, gates, ress, ys, hs;
  int32_t rows, cols;
  float eps;
};
hipError_t launch_join_fwd(const JoinFwdArgs& a, int dtype, hipStream_t s);

struct JoinBwdArgs {
  const void* x;
  const void* gate;     // or null
  const void* h;
  const void* y_bar;
  const void* h_bar;    // or null: zeros
  const float* stats;
  const float* w1;
  const float* b1;
  const float* scale;
  const float* w2;
  void* x_bar;          // each of these or null
  void* gate_bar;
  void* res_bar;
  float* bar[5];        // w1, b1, scale, w2, b2; each or null
  float* part;          // [parts][5][cols] (none needed for one part)
  float* means;         // [rows][2] for rows that do not fit registers, or null
  int64_t xs, gates, hs, ybs, hbs, xbs, gbs, rbs;
  int32_t rows, cols, parts;
  bool sums;            // any of bar
};
int join_parts(int32_t rows, int32_t cols);
bool join_means(int32_t cols);
// The kernel and, with sums in more than one part, the launch that adds them in a fixed order.
hipError_t launch_join_bwd(const JoinBwdArgs& a, int dtype, hipStream_t s);

}  // namespace etpc
