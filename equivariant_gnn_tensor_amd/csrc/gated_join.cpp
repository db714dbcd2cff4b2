// C ABI of the gated join between two norms: argument checks on the host, then its launches.
#include "gated_join_args.hpp"
#include "kernels.hpp"
#include "operands.hpp"
#include "profile.hpp"

namespace etpc {
namespace {

// Regions of the backward pass's workspace in floats: partial sums, then the rows' means.
struct JoinSpace {
  int64_t part, means;
  size_t bytes() const { return static_cast<size_t>(part + means) * sizeof(float); }
};
JoinSpace join_space(int64_t rows, int64_t cols) {
  const int parts = join_parts(static_cast<int32_t>(rows), static_cast<int32_t>(cols));
  return JoinSpace{parts > 1 ? int64_t{5} * parts * cols : 0, join_means(static_cast<int32_t>(cols)) ? 2 * rows : 0};
}

}  // namespace
}  // namespace etpc

using namespace etpc;

extern "C" {

etpc_status etpc_norm_gate_add_norm(int64_t n_rows, int64_t n_cols, int32_t dtype, const void* x, int64_t x_stride,
                                    const void* gate, int64_t gate_stride, const void* residual, int64_t residual_stride,
                                    const float* w1, const float* b1, const float* scale, const float* w2,
                                    const float* b2, float eps, void* y, int64_t y_stride, void* h, int64_t h_stride,
                                    float* stats, hipStream_t s) {
  ETPC_TRY(check_sizes(n_rows, n_cols, dtype));
  ETPC_TRY(check_eps(eps));
  if (n_cols < 1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "a row needs at least one column");
  if (n_rows == 0) return ETPC_OK;
  const Mat mx{"x", x, x_stride}, mg{"gate", gate, gate_stride}, mr{"residual", residual, residual_stride},
      my{"y", y, y_stride}, mh{"h", h, h_stride};
  ETPC_TRY(check_mat(mx, n_rows, n_cols, dtype, false));
  if (gate != nullptr) ETPC_TRY(check_mat(mg, n_rows, n_cols, dtype, false));
  if (residual != nullptr) ETPC_TRY(check_mat(mr, n_rows, n_cols, dtype, false));
  ETPC_TRY(check_mat(my, n_rows, n_cols, dtype, true));
  if (h != nullptr) ETPC_TRY(check_mat(mh, n_rows, n_cols, dtype, true));
  const int64_t size = size_of(dtype);
  const Operand o1{"w1", w1, 4 * n_cols}, o2{"b1", b1, 4 * n_cols}, o3{"scale", scale, 4 * n_cols},
      o4{"w2", w2, 4 * n_cols}, o5{"b2", b2, 4 * n_cols}, os{"stats", stats, 16 * n_rows};
  ETPC_TRY(check_floats({o1, o2, o3, o4, o5, os}));
  ETPC_TRY(check_apart({{my, n_rows, n_cols, size}, {mh, n_rows, n_cols, size}, os},
                       {{mx, n_rows, n_cols, size}, {mg, n_rows, n_cols, size}, {mr, n_rows, n_cols, size}, o1, o2, o3, o4,
                        o5}));
  JoinFwdArgs a{};
  a.x = x, a.gate = gate, a.res = residual, a.w1 = w1, a.b1 = b1, a.scale = scale, a.w2 = w2, a.b2 = b2;
  a.y = y, a.h = h, a.stats = stats;
  a.xs = x_stride, a.gates = gate_stride, a.ress = residual_stride, a.ys = y_stride, a.hs = h_stride;
  a.rows = static_cast<int32_t>(n_rows), a.cols = static_cast<int32_t>(n_cols), a.eps = eps;
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_join_fwd(a, dtype, s));
  return ETPC_OK;
}

etpc_status etpc_norm_gate_add_norm_workspace_size(int64_t n_rows, int64_t n_cols, size_t* bytes) {
  if (bytes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null output");
  ETPC_TRY(check_sizes(n_rows, n_cols, ETPC_F32));
  *bytes = n_rows > 0 && n_cols > 0 ? join_space(n_rows, n_cols).bytes() : 0;
  return ETPC_OK;
}

etpc_status etpc_norm_gate_add_norm_backward(
    int64_t n_rows, int64_t n_cols, int32_t dtype, const void* x, int64_t x_stride, const void* gate,
    int64_t gate_stride, const void* h, int64_t h_stride, const void* y_bar, int64_t y_bar_stride, const void* h_bar,
    int64_t h_bar_stride, const float* stats, const float* w1, const float* b1, const float* scale, const float* w2,
    void* x_bar, int64_t x_bar_stride, void* gate_bar, int64_t gate_bar_stride, void* residual_bar,
    int64_t residual_bar_stride, float* w1_bar, float* b1_bar, float* scale_bar, float* w2_bar, float* b2_bar, void* ws,
    size_t ws_bytes, hipStream_t s) {
  ETPC_TRY(check_sizes(n_rows, n_cols, dtype));
  if (n_cols < 1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "a row needs at least one column");
  if (gate == nullptr && gate_bar != nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "gate_bar without a gate");
  JoinBwdArgs a{};
  float* const bars[5] = {w1_bar, b1_bar, scale_bar, w2_bar, b2_bar};
  for (int j = 0; j < 5; ++j) a.bar[j] = bars[j], a.sums = a.sums || bars[j] != nullptr;
  const Operand p1{"w1_bar", w1_bar, 4 * n_cols}, p2{"b1_bar", b1_bar, 4 * n_cols}, p3{"scale_bar", scale_bar, 4 * n_cols},
      p4{"w2_bar", w2_bar, 4 * n_cols}, p5{"b2_bar", b2_bar, 4 * n_cols};
  ETPC_TRY(check_floats({p1, p2, p3, p4, p5}));
  if (n_rows == 0) {
    ETPC_TRY(check_apart({p1, p2, p3, p4, p5}, {}));
    for (float* bar : bars)
      if (bar != nullptr) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_fill(bar, n_cols, 0.f, s));
    return ETPC_OK;
  }
  const Mat mx{"x", x, x_stride}, mg{"gate", gate, gate_stride}, mh{"h", h, h_stride}, my{"y_bar", y_bar, y_bar_stride},
      mhb{"h_bar", h_bar, h_bar_stride}, mxb{"x_bar", x_bar, x_bar_stride}, mgb{"gate_bar", gate_bar, gate_bar_stride},
      mrb{"residual_bar", residual_bar, residual_bar_stride};
  ETPC_TRY(check_mat(mx, n_rows, n_cols, dtype, false));
  if (gate != nullptr) ETPC_TRY(check_mat(mg, n_rows, n_cols, dtype, false));
  ETPC_TRY(check_mat(mh, n_rows, n_cols, dtype, false));
  ETPC_TRY(check_mat(my, n_rows, n_cols, dtype, false));
  if (h_bar != nullptr) ETPC_TRY(check_mat(mhb, n_rows, n_cols, dtype, false));
  if (x_bar != nullptr) ETPC_TRY(check_mat(mxb, n_rows, n_cols, dtype, true));
  if (gate_bar != nullptr) ETPC_TRY(check_mat(mgb, n_rows, n_cols, dtype, true));
  if (residual_bar != nullptr) ETPC_TRY(check_mat(mrb, n_rows, n_cols, dtype, true));
  if (stats == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null stats");
  const JoinSpace space = join_space(n_rows, n_cols);
  if (a.sums) ETPC_TRY(check_parts(ws, ws_bytes, space.bytes()));
  const int64_t size = size_of(dtype);
  const Operand o1{"w1", w1, 4 * n_cols}, o2{"b1", b1, 4 * n_cols}, o3{"scale", scale, 4 * n_cols},
      o4{"w2", w2, 4 * n_cols}, os{"stats", stats, 16 * n_rows};
  ETPC_TRY(check_floats({o1, o2, o3, o4, os}));
  ETPC_TRY(check_apart({{mxb, n_rows, n_cols, size}, {mgb, n_rows, n_cols, size}, {mrb, n_rows, n_cols, size}, p1, p2, p3, p4,
                        p5, {"the workspace", a.sums ? ws : nullptr, static_cast<int64_t>(space.bytes())}},
                       {{mx, n_rows, n_cols, size}, {mg, n_rows, n_cols, size}, {mh, n_rows, n_cols, size},
                        {my, n_rows, n_cols, size}, {mhb, n_rows, n_cols, size}, o1, o2, o3, o4, os}));
  if (!a.sums && x_bar == nullptr && gate_bar == nullptr && residual_bar == nullptr) return ETPC_OK;
  a.x = x, a.gate = gate, a.h = h, a.y_bar = y_bar, a.h_bar = h_bar, a.stats = stats;
  a.w1 = w1, a.b1 = b1, a.scale = scale, a.w2 = w2;
  a.x_bar = x_bar, a.gate_bar = gate_bar, a.res_bar = residual_bar;
  a.part = static_cast<float*>(ws);
  if (a.sums && space.means > 0) a.means = a.part + space.part;
  a.xs = x_stride, a.gates = gate_stride, a.hs = h_stride, a.ybs = y_bar_stride, a.hbs = h_bar_stride;
  a.xbs = x_bar_stride, a.gbs = gate_bar_stride, a.rbs = residual_bar_stride;
  a.rows = static_cast<int32_t>(n_rows), a.cols = static_cast<int32_t>(n_cols);
  a.parts = join_parts(a.rows, a.cols);
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_join_bwd(a, dtype, s));
  return ETPC_OK;
}

}  // extern "C"
