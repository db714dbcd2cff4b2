// C ABI of the node-wise operators: argument checks on the host, then one or two launches.
#include <cmath>

#include "kernels.hpp"
#include "nodewise.hpp"
#include "operands.hpp"
#include "profile.hpp"

namespace etpc {
namespace {

constexpr int64_t kMaxDim = int64_t{1} << 20;

etpc_status make_drop(const etpc_dropout_spec* d, DropArgs* out) {
  *out = DropArgs{};
  if (d == nullptr) return ETPC_OK;
  if (!(d->p >= 0.0 && d->p <= 1.0)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "dropout probability must be in [0, 1]");
  if (reinterpret_cast<uintptr_t>(d->offset_add) % sizeof(uint64_t) != 0)
    ETPC_FAIL(ETPC_ERR_INVALID_ARG, "offset_add is not aligned to its element");
  const uint32_t t = static_cast<uint32_t>(std::nearbyint(65536.0 * d->p));
  out->threshold = t;
  out->scale = t < 65536u ? static_cast<float>(65536.0 / (65536.0 - t)) : 0.f;
  out->seed = d->seed;
  out->offset = d->offset;
  out->offset_add = d->offset_add;
  return ETPC_OK;
}

etpc_status norm_forward(int64_t rows, int64_t cols, int32_t dtype, const Mat& x, const Mat& res,
                         const etpc_dropout_spec* drop, const float* w, const float* b, float eps, const Mat& y,
                         const Mat& h, float* mean, float* rstd, hipStream_t s) {
  ETPC_TRY(check_sizes(rows, cols, dtype));
  ETPC_TRY(check_eps(eps));
  if (cols < 1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "a row needs at least one column");
  NormFwdArgs a{};
  ETPC_TRY(make_drop(drop, &a.drop));
  if (rows == 0) return ETPC_OK;
  ETPC_TRY(check_mat(x, rows, cols, dtype, false));
  if (res.p != nullptr) ETPC_TRY(check_mat(res, rows, cols, dtype, false));
  ETPC_TRY(check_mat(y, rows, cols, dtype, true));
  if (h.p != nullptr) ETPC_TRY(check_mat(h, rows, cols, dtype, true));
  const int64_t size = size_of(dtype);
  const Operand ow{"w", w, 4 * cols}, ob{"b", b, 4 * cols}, om{"mean", mean, 4 * rows}, os{"rstd", rstd, 4 * rows};
  ETPC_TRY(check_floats({ow, ob, om, os}));
  ETPC_TRY(check_apart({{y, rows, cols, size}, {h, rows, cols, size}, om, os},
                       {{x, rows, cols, size}, {res, rows, cols, size}, ow, ob, {"offset_add", a.drop.offset_add, 8}}));
  a.x = x.p, a.res = res.p, a.w = w, a.b = b;
  a.y = const_cast<void*>(y.p), a.h = const_cast<void*>(h.p), a.mean = mean, a.rstd = rstd;
  a.xs = x.stride, a.ress = res.stride, a.ys = y.stride, a.hs = h.stride;
  a.rows = static_cast<int32_t>(rows), a.cols = static_cast<int32_t>(cols), a.eps = eps;
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_norm_fwd(a, dtype, s));
  return ETPC_OK;
}

etpc_status norm_backward(int64_t rows, int64_t cols, int32_t dtype, const Mat& h, const Mat& y_bar, const Mat& h_bar,
                          const float* mean, const float* rstd, const float* w, const etpc_dropout_spec* drop,
                          const Mat& x_bar, const Mat& res_bar, float* w_bar, float* b_bar, void* ws, size_t ws_bytes,
                          hipStream_t s) {
  ETPC_TRY(check_sizes(rows, cols, dtype));
  if (cols < 1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "a row needs at least one column");
  NormBwdArgs a{};
  ETPC_TRY(make_drop(drop, &a.drop));
  if (rows == 0) {
    if (w_bar != nullptr) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_fill(w_bar, cols, 0.f, s));
    if (b_bar != nullptr) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_fill(b_bar, cols, 0.f, s));
    return ETPC_OK;
  }
  ETPC_TRY(check_mat(h, rows, cols, dtype, false));
  ETPC_TRY(check_mat(y_bar, rows, cols, dtype, false));
  if (h_bar.p != nullptr) ETPC_TRY(check_mat(h_bar, rows, cols, dtype, false));
  if (x_bar.p != nullptr) ETPC_TRY(check_mat(x_bar, rows, cols, dtype, true));
  if (res_bar.p != nullptr) ETPC_TRY(check_mat(res_bar, rows, cols, dtype, true));
  if (mean == nullptr || rstd == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null mean or rstd");
  a.rows = static_cast<int32_t>(rows), a.cols = static_cast<int32_t>(cols);
  const bool sums = w_bar != nullptr || b_bar != nullptr;
  const size_t need = sums ? parts_bytes(norm_parts_most(a.rows, a.cols), 2 * cols) : 0;
  if (sums) ETPC_TRY(check_parts(ws, ws_bytes, need));
  const int64_t size = size_of(dtype);
  const Operand ow{"w", w, 4 * cols}, om{"mean", mean, 4 * rows}, os{"rstd", rstd, 4 * rows},
      owb{"w_bar", w_bar, 4 * cols}, obb{"b_bar", b_bar, 4 * cols};
  ETPC_TRY(check_floats({ow, om, os, owb, obb}));
  ETPC_TRY(check_apart({{x_bar, rows, cols, size}, {res_bar, rows, cols, size}, owb, obb,
                        {"the workspace", ws, static_cast<int64_t>(need)}},
                       {{h, rows, cols, size}, {y_bar, rows, cols, size}, {h_bar, rows, cols, size}, ow, om, os,
                        {"offset_add", a.drop.offset_add, 8}}));
  if (!sums && x_bar.p == nullptr && res_bar.p == nullptr) return ETPC_OK;
  a.h = h.p, a.y_bar = y_bar.p, a.h_bar = h_bar.p, a.mean = mean, a.rstd = rstd, a.w = w;
  a.x_bar = const_cast<void*>(x_bar.p), a.res_bar = const_cast<void*>(res_bar.p), a.w_bar = w_bar, a.b_bar = b_bar;
  a.part = static_cast<float*>(ws);
  a.hs = h.stride, a.ybs = y_bar.stride, a.hbs = h_bar.stride, a.xbs = x_bar.stride, a.rbs = res_bar.stride;
  a.parts = norm_parts(a, dtype);
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_norm_bwd(a, dtype, s));
  if (sums && a.parts > 1)
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_parts_reduce(a.part, a.parts, a.cols, w_bar, b_bar, s));
  return ETPC_OK;
}

etpc_status make_table(int32_t n, const etpc_irrep* irreps, IrrepTable* t) {
  if (n < 0 || (n > 0 && irreps == nullptr)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null or negative irreps");
  if (n > kMaxIrreps) ETPC_FAIL(ETPC_ERR_UNSUPPORTED, "at most 64 irreps blocks");
  int64_t dim = 0, channels = 0, biases = 0, groups = 0;
  t->n = n;
  for (int32_t k = 0; k < n; ++k) {
    const etpc_irrep& ir = irreps[k];
    if (ir.mul < 1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "irreps multiplicity must be at least 1");
    if (ir.l < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative degree");
    if (ir.l > kMaxL) ETPC_FAIL(ETPC_ERR_UNSUPPORTED, "irreps degree above 3");
    if (ir.parity != 1 && ir.parity != -1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "parity must be 1 or -1");
    const bool bias = ir.l == 0 && ir.parity == 1;
    t->blk[k] = IrrepBlock{static_cast<int32_t>(dim), ir.mul, ir.l, static_cast<int32_t>(channels),
                           bias ? static_cast<int32_t>(biases) : -1, static_cast<int32_t>(groups), 0, 0};
    dim += static_cast<int64_t>(ir.mul) * (2 * ir.l + 1);
    channels += ir.mul;
    biases += bias ? ir.mul : 0;
    groups += (ir.mul + int64_t{7}) / 8;
    // a workgroup's 256 rows are addressed by 32-bit byte offsets
    if (dim > kMaxDim) ETPC_FAIL(ETPC_ERR_OVERFLOW, "feature rows must be at most 2^20 wide");
  }
  t->dim = static_cast<int32_t>(dim);
  t->channels = static_cast<int32_t>(channels);
  t->biases = static_cast<int32_t>(biases);
  return ETPC_OK;
}

Mat features(const char* name, const float* p, const IrrepTable& t) { return Mat{name, p, t.dim}; }
Operand features(const Mat& m, int64_t n_nodes, const IrrepTable& t) {
  return Operand{m.name, m.p, n_nodes * t.dim * int64_t{4}};
}
Operand floats(const char* name, const float* p, int64_t n) { return Operand{name, p, 4 * n}; }

}  // namespace
}  // namespace etpc

using namespace etpc;

extern "C" {

etpc_status etpc_dropout(int64_t n_rows, int64_t n_cols, int32_t dtype, const void* x, int64_t x_stride,
                         const etpc_dropout_spec* drop, void* y, int64_t y_stride, hipStream_t s) {
  ETPC_TRY(check_sizes(n_rows, n_cols, dtype));
  if (drop == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null dropout spec");
  DropArgs d;
  ETPC_TRY(make_drop(drop, &d));
  if (n_rows == 0 || n_cols == 0) return ETPC_OK;
  const Mat in{"x", x, x_stride}, out{"y", y, y_stride};
  ETPC_TRY(check_mat(in, n_rows, n_cols, dtype, false));
  ETPC_TRY(check_mat(out, n_rows, n_cols, dtype, true));
  const bool in_place = x == y && (n_rows == 1 || x_stride == y_stride);
  const Operand src{in, n_rows, n_cols, size_of(dtype)}, dst{out, n_rows, n_cols, size_of(dtype)};
  if (!in_place) ETPC_TRY(check_apart({dst}, {src}));
  ETPC_TRY(check_apart({dst}, {{"offset_add", d.offset_add, 8}}));
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_dropout(x, x_stride, y, y_stride, static_cast<int32_t>(n_rows),
                                                 static_cast<int32_t>(n_cols), dtype, d, s));
  return ETPC_OK;
}

etpc_status etpc_layer_norm(int64_t n_rows, int64_t n_cols, int32_t dtype, const void* x, int64_t x_stride,
                            const float* w, const float* b, float eps, void* y, int64_t y_stride, float* mean,
                            float* rstd, hipStream_t s) {
  return norm_forward(n_rows, n_cols, dtype, Mat{"x", x, x_stride}, Mat{"residual", nullptr, 0}, nullptr, w, b, eps,
                      Mat{"y", y, y_stride}, Mat{"h", nullptr, 0}, mean, rstd, s);
}

etpc_status etpc_layer_norm_workspace_size(int64_t n_rows, int64_t n_cols, size_t* bytes) {
  if (bytes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null output");
  ETPC_TRY(check_sizes(n_rows, n_cols, ETPC_F32));
  *bytes = n_rows > 0 && n_cols > 0
               ? parts_bytes(norm_parts_most(static_cast<int32_t>(n_rows), static_cast<int32_t>(n_cols)), 2 * n_cols)
               : 0;
  return ETPC_OK;
}

etpc_status etpc_layer_norm_backward(int64_t n_rows, int64_t n_cols, int32_t dtype, const void* x, int64_t x_stride,
                                     const void* y_bar, int64_t y_bar_stride, const float* mean, const float* rstd,
                                     const float* w, void* x_bar, int64_t x_bar_stride, float* w_bar, float* b_bar,
                                     void* ws, size_t ws_bytes, hipStream_t s) {
  return norm_backward(n_rows, n_cols, dtype, Mat{"x", x, x_stride}, Mat{"y_bar", y_bar, y_bar_stride},
                       Mat{"h_bar", nullptr, 0}, mean, rstd, w, nullptr, Mat{"x_bar", x_bar, x_bar_stride},
                       Mat{"residual_bar", nullptr, 0}, w_bar, b_bar, ws, ws_bytes, s);
}

etpc_status etpc_dropout_add_layer_norm(int64_t n_rows, int64_t n_cols, int32_t dtype, const void* x, int64_t x_stride,
                                        const void* residual, int64_t residual_stride, const etpc_dropout_spec* drop,
                                        const float* w, const float* b, float eps, void* y, int64_t y_stride, void* h,
                                        int64_t h_stride, float* mean, float* rstd, hipStream_t s) {
  return norm_forward(n_rows, n_cols, dtype, Mat{"x", x, x_stride}, Mat{"residual", residual, residual_stride}, drop,
                      w, b, eps, Mat{"y", y, y_stride}, Mat{"h", h, h_stride}, mean, rstd, s);
}

etpc_status etpc_dropout_add_layer_norm_backward(int64_t n_rows, int64_t n_cols, int32_t dtype, const void* h,
                                                 int64_t h_stride, const void* y_bar, int64_t y_bar_stride,
                                                 const void* h_bar, int64_t h_bar_stride, const float* mean,
                                                 const float* rstd, const float* w, const etpc_dropout_spec* drop,
                                                 void* x_bar, int64_t x_bar_stride, void* residual_bar,
                                                 int64_t residual_bar_stride, float* w_bar, float* b_bar, void* ws,
                                                 size_t ws_bytes, hipStream_t s) {
  return norm_backward(n_rows, n_cols, dtype, Mat{"h", h, h_stride}, Mat{"y_bar", y_bar, y_bar_stride},
                       Mat{"h_bar", h_bar, h_bar_stride}, mean, rstd, w, drop, Mat{"x_bar", x_bar, x_bar_stride},
                       Mat{"residual_bar", residual_bar, residual_bar_stride}, w_bar, b_bar, ws, ws_bytes, s);
}

etpc_status etpc_irreps_dims(int32_t n_blocks, const etpc_irrep* irreps, int64_t* dim, int64_t* channels,
                             int64_t* biases) {
  IrrepTable t;
  ETPC_TRY(make_table(n_blocks, irreps, &t));
  if (dim != nullptr) *dim = t.dim;
  if (channels != nullptr) *channels = t.channels;
  if (biases != nullptr) *biases = t.biases;
  return ETPC_OK;
}

etpc_status etpc_irreps_dropout(int32_t n_blocks, const etpc_irrep* irreps, int32_t n_nodes, const float* x,
                                const etpc_dropout_spec* drop, float* y, hipStream_t s) {
  IrrepTable t;
  ETPC_TRY(make_table(n_blocks, irreps, &t));
  if (n_nodes < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative n_nodes");
  if (drop == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null dropout spec");
  DropArgs d;
  ETPC_TRY(make_drop(drop, &d));
  if (n_nodes == 0 || t.n == 0) return ETPC_OK;
  const Mat mx = features("x", x, t), my = features("y", y, t);
  ETPC_TRY(check_mat(mx, n_nodes, t.dim, ETPC_F32, false));
  ETPC_TRY(check_mat(my, n_nodes, t.dim, ETPC_F32, true));
  if (x != y) ETPC_TRY(check_apart({features(my, n_nodes, t)}, {features(mx, n_nodes, t)}));
  ETPC_TRY(check_apart({features(my, n_nodes, t)}, {{"offset_add", d.offset_add, 8}}));
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_irreps_dropout(t, x, y, n_nodes, d, s));
  return ETPC_OK;
}

etpc_status etpc_irreps_norm(int32_t n_blocks, const etpc_irrep* irreps, int32_t n_nodes, const float* x,
                             const float* w, const float* b, float eps, float* y, float* stats, hipStream_t s) {
  IrrepTable t;
  ETPC_TRY(make_table(n_blocks, irreps, &t));
  ETPC_TRY(check_eps(eps));
  if (n_nodes < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative n_nodes");
  if (n_nodes == 0 || t.n == 0) return ETPC_OK;
  const Mat mx = features("x", x, t), my = features("y", y, t);
  ETPC_TRY(check_mat(mx, n_nodes, t.dim, ETPC_F32, false));
  ETPC_TRY(check_mat(my, n_nodes, t.dim, ETPC_F32, true));
  const Operand ow = floats("w", w, t.channels), ob = floats("b", b, t.biases),
                os = floats("stats", stats, int64_t{2} * n_nodes * t.n);
  ETPC_TRY(check_floats({ow, ob, os}));
  ETPC_TRY(check_apart({features(my, n_nodes, t), os}, {features(mx, n_nodes, t), ow, ob}));
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_irreps_norm_fwd(t, x, w, b, eps, y, stats, n_nodes, s));
  return ETPC_OK;
}

etpc_status etpc_irreps_norm_workspace_size(int32_t n_blocks, const etpc_irrep* irreps, int32_t n_nodes,
                                            size_t* bytes) {
  if (bytes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null output");
  IrrepTable t;
  ETPC_TRY(make_table(n_blocks, irreps, &t));
  if (n_nodes < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative n_nodes");
  *bytes = n_nodes > 0 && t.n > 0 ? static_cast<size_t>(irreps_norm_part_floats(t, n_nodes)) * sizeof(float) : 0;
  return ETPC_OK;
}

etpc_status etpc_irreps_norm_backward(int32_t n_blocks, const etpc_irrep* irreps, int32_t n_nodes, const float* x,
                                      const float* y_bar, const float* stats, const float* w, float* x_bar,
                                      float* w_bar, float* b_bar, void* ws, size_t ws_bytes, hipStream_t s) {
  IrrepTable t;
  ETPC_TRY(make_table(n_blocks, irreps, &t));
  if (n_nodes < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative n_nodes");
  if (t.n == 0) return ETPC_OK;
  if (t.biases == 0) b_bar = nullptr;
  if (n_nodes == 0) {
    if (w_bar != nullptr) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_fill(w_bar, t.channels, 0.f, s));
    if (b_bar != nullptr) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_fill(b_bar, t.biases, 0.f, s));
    return ETPC_OK;
  }
  const Mat mx = features("x", x, t), my = features("y_bar", y_bar, t), mo = features("x_bar", x_bar, t);
  ETPC_TRY(check_mat(mx, n_nodes, t.dim, ETPC_F32, false));
  ETPC_TRY(check_mat(my, n_nodes, t.dim, ETPC_F32, false));
  if (x_bar != nullptr) ETPC_TRY(check_mat(mo, n_nodes, t.dim, ETPC_F32, true));
  if (stats == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null stats");
  const bool sums = w_bar != nullptr || b_bar != nullptr;
  const int64_t part_floats = sums ? irreps_norm_part_floats(t, n_nodes) : 0;
  if (sums) ETPC_TRY(check_parts(ws, ws_bytes, static_cast<size_t>(part_floats) * sizeof(float)));
  const Operand ow = floats("w", w, t.channels), os = floats("stats", stats, int64_t{2} * n_nodes * t.n),
                owb = floats("w_bar", w_bar, t.channels), obb = floats("b_bar", b_bar, t.biases);
  ETPC_TRY(check_floats({ow, os, owb, obb}));
  ETPC_TRY(check_apart({features(mo, n_nodes, t), owb, obb, floats("the workspace", static_cast<const float*>(ws), part_floats)},
                       {features(mx, n_nodes, t), features(my, n_nodes, t), ow, os}));
  if (!sums && x_bar == nullptr) return ETPC_OK;
  float* part = static_cast<float*>(ws);
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_irreps_norm_bwd(t, x, y_bar, stats, w, x_bar, w_bar, b_bar, part, n_nodes, s));
  return ETPC_OK;
}

}  // extern "C"
