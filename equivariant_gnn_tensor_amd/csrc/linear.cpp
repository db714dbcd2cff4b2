// C ABI of the dense layer: argument checks on the host, then its launches.
#include <algorithm>

#include "kernels.hpp"
#include "linear.hpp"
#include "narrow_args.hpp"
#include "operands.hpp"
#include "profile.hpp"

namespace etpc {
namespace {

etpc_status check_layer(int64_t rows, int64_t n_in, int64_t n_out, int32_t dtype, int32_t act) {
  ETPC_TRY(check_sizes(rows, std::max(n_in, n_out), dtype));
  if (n_in < 1 || n_out < 1) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "a layer needs at least one input and one output");
  constexpr int64_t most = (int64_t{1} << 56) - 1;   // sizes in bytes and partial sums stay within 63 bits
  if (rows > 0 && (n_in > most / rows || n_out > most / rows)) ETPC_FAIL(ETPC_ERR_OVERFLOW, "rows times columns must be < 2^56");
  if (n_in > most / n_out) ETPC_FAIL(ETPC_ERR_OVERFLOW, "n_in times n_out must be < 2^56");
  if (act < ETPC_ACT_NONE || act > ETPC_ACT_TANH) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "bad activation");
  return ETPC_OK;
}

// A weight matrix [n_in][n_out] with either axis contiguous, as rows of the contiguous one.
struct Weights {
  Mat m;
  int64_t rows, cols;
  bool by_out;   // rows of n_out numbers, one for each input
};
etpc_status make_weights(const char* name, const void* p, int64_t in_stride, int64_t out_stride, int64_t n_in,
                         int64_t n_out, int32_t dtype, bool output, Weights* w) {
  w->by_out = out_stride == 1 || n_out == 1;
  if (!w->by_out && in_stride != 1 && n_in != 1)
    ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string(name) + ": one of the strides must be 1");
  w->m = Mat{name, p, w->by_out ? in_stride : out_stride};
  w->rows = w->by_out ? n_in : n_out;
  w->cols = w->by_out ? n_out : n_in;
  return check_mat(w->m, w->rows, w->cols, dtype, output);
}
Operand operand(const Weights& w, int64_t size) { return Operand{w.m, w.rows, w.cols, size}; }

// Regions of the backward pass's workspace, each a multiple of 256 bytes.
struct LinearSpace {
  size_t z_bar, w_part, b_part, x_part, bytes;
  int64_t z_bar_stride;
};
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Weight gradient as a product: rows of the contiguous axis of w_bar by the other.
MatmulArgs weight_product(int64_t rows, int64_t n_in, int64_t n_out, bool by_out) {
  MatmulArgs a{};
  a.M = static_cast<int32_t>(by_out ? n_in : n_out);
  a.N = static_cast<int32_t>(by_out ? n_out : n_in);
  a.K = static_cast<int32_t>(rows);
  return a;
}

// Partial sums of a layer's product [rows][k] x [k][cols], when it is split: the same whatever the layout.
size_t product_space(int64_t rows, int64_t k, int64_t cols, int32_t dtype) {
  MatmulArgs a{};
  a.M = static_cast<int32_t>(rows), a.N = static_cast<int32_t>(cols), a.K = static_cast<int32_t>(k);
  const int splits = matmul_shape(a, MatmulForm::kRowsCols, dtype, false).splits;
  return splits > 1 ? round256(static_cast<size_t>(splits) * static_cast<size_t>(rows * cols) * sizeof(float)) : 0;
}
size_t forward_space(int64_t rows, int64_t n_in, int64_t n_out, int32_t dtype) {
  return narrow::fits_fwd(rows, n_in, n_out, dtype) ? 0 : product_space(rows, n_in, n_out, dtype);
}

// Whether one or two rows past the last whole tile are better left to the kernel for few rows (from three on
// it is slower than a tile).  They are where some CUs would work one tile longer because of them, for
// longer than that kernel's launch takes.  fp32 tiles are bound by a CU's matrix cores, so tiles that are resident
// together count one after another; 16-bit ones overlap.  A slice of a 64 x 64 tile is 0.45 us of a CU in fp32,
// 0.07 in 16 bits.  150 sizes with a remainder of one or two rows, with and without: 4097 x 2047 -> 511 fp32 80 us
// and 104, 16386 x 1024 -> 136 77 and 124, 4097 x 512 -> 256 17.5 and 20.9, 8194 x 256 -> 256 18 and 18, 6146 x
// 136 -> 512 18.6 and 16.6; 8193 x 2048 -> 2048 bf16 70 and 95, 16385 x 256 -> 2048 33 and 37, 16385 x 64 -> 2048 25 and
// 25, and 8194 x 4096 -> 512, whose tiles are all resident, 60 and 53.
bool rows_apart(const MatmulArgs& a, const MatmulShape& shape, int32_t dtype) {
  const int32_t over = a.M % shape.tile;
  if (over == 0 || over > kFewRows || a.M == over) return false;
  const int64_t across = (a.N + shape.tile - 1) / shape.tile, down = a.M / shape.tile;
  const int64_t resident = matmul_resident(shape.tile, shape.stages);
  const auto rounds = [&](int64_t tiles) {
    const int64_t all = (tiles + kCus * resident - 1) / (kCus * resident);
    return dtype != ETPC_F32 ? all : all > 1 ? all * resident : (tiles + kCus - 1) / kCus;
  };
  const double side = shape.tile / 64, slices = static_cast<double>(a.K) * static_cast<double>(size_of(dtype)) / 128;
  const double round = slices * side * side * (dtype == ETPC_F32 ? 0.45 : 0.07);
  return static_cast<double>(rounds((down + 1) * across) - rounds(down * across)) * round > 4.0;
}

// A layer's product, split when its shape is.
hipError_t run_product(MatmulArgs a, MatmulForm form, int32_t dtype, void* space, hipStream_t s) {
  const MatmulShape shape = matmul_shape(a, form, dtype, false);
  if (shape.splits > 1) {
    a.part = static_cast<float*>(space);
    const hipError_t e = launch_matmul(a, form, dtype, shape, s);
    a.splits = shape.splits;
    return e != hipSuccess ? e : launch_layer_parts(a, dtype, s);
  }
  if (!rows_apart(a, shape, dtype)) return launch_matmul(a, form, dtype, shape, s);
  const int32_t over = a.M % shape.tile, whole = a.M - over;
  const int64_t size = size_of(dtype);
  const auto from = [&](const void* p, int64_t stride) { return p == nullptr ? p : static_cast<const char*>(p) + whole * stride * size; };
  MatmulArgs rest = a;
  rest.M = over;
  rest.a = from(a.a, a.lda), rest.res = from(a.res, a.ldres);
  rest.c = const_cast<void*>(from(a.c, a.ldc)), rest.z = const_cast<void*>(from(a.z, a.ldz));
  a.M = whole;
  const hipError_t e = launch_matmul(a, form, dtype, shape, s);
  return e != hipSuccess ? e : launch_matmul(rest, form, dtype, matmul_shape(rest, form, dtype, false), s);
}

// The same whatever the layout of w, the addresses and the wanted outputs.
LinearSpace linear_space(int64_t rows, int64_t n_in, int64_t n_out, int32_t dtype, int32_t act) {
  LinearSpace s{};
  if (narrow::fits_bwd(rows, n_in, n_out, dtype)) {
    s.b_part = round256(static_cast<size_t>(narrow::bwd_groups(rows)) * static_cast<size_t>(n_in * n_out + n_out) * sizeof(float));
    s.bytes = s.b_part;
    return s;
  }
  const int64_t size = size_of(dtype);
  s.z_bar_stride = (n_out + 7) / 8 * 8;
  s.z_bar = act != ETPC_ACT_NONE ? round256(static_cast<size_t>(rows * s.z_bar_stride * size)) : 0;
  const MatmulArgs a = weight_product(rows, n_in, n_out, true), b = weight_product(rows, n_in, n_out, false);
  const int splits = std::max(matmul_shape(a, MatmulForm::kColsCols, dtype, true).splits,
                              matmul_shape(b, MatmulForm::kColsCols, dtype, true).splits);
  s.w_part = splits > 1 ? round256(static_cast<size_t>(splits) * static_cast<size_t>(n_in * n_out) * sizeof(float)) : 0;
  const int parts = slope_parts(static_cast<int32_t>(rows), static_cast<int32_t>(n_out));
  s.b_part = round256(static_cast<size_t>(parts) * static_cast<size_t>(n_out) * sizeof(float));
  s.x_part = product_space(rows, n_out, n_in, dtype);
  s.bytes = s.z_bar + s.w_part + s.b_part + s.x_part;
  return s;
}

}  // namespace
}  // namespace etpc

using namespace etpc;

extern "C" {

etpc_status etpc_linear(int64_t n_rows, int64_t n_in, int64_t n_out, int32_t dtype, const void* x, int64_t x_stride,
                        const void* w, int64_t w_in_stride, int64_t w_out_stride, const float* b, const void* residual,
                        int64_t residual_stride, int32_t act, void* y, int64_t y_stride, void* z, int64_t z_stride,
                        void* ws, size_t ws_bytes, hipStream_t s) {
  ETPC_TRY(check_layer(n_rows, n_in, n_out, dtype, act));
  if (n_rows == 0) return ETPC_OK;
  const int64_t size = size_of(dtype);
  const Mat mx{"x", x, x_stride}, mr{"residual", residual, residual_stride}, my{"y", y, y_stride}, mz{"z", z, z_stride};
  ETPC_TRY(check_mat(mx, n_rows, n_in, dtype, false));
  Weights mw;
  ETPC_TRY(make_weights("w", w, w_in_stride, w_out_stride, n_in, n_out, dtype, false, &mw));
  if (residual != nullptr) ETPC_TRY(check_mat(mr, n_rows, n_out, dtype, false));
  ETPC_TRY(check_mat(my, n_rows, n_out, dtype, true));
  if (z != nullptr) ETPC_TRY(check_mat(mz, n_rows, n_out, dtype, true));
  const Operand ob{"b", b, 4 * n_out};
  ETPC_TRY(check_floats({ob}));
  const size_t need = forward_space(n_rows, n_in, n_out, dtype);
  ETPC_TRY(check_parts(ws, ws_bytes, need));
  ETPC_TRY(check_apart({{my, n_rows, n_out, size}, {mz, n_rows, n_out, size},
                        {"the workspace", need > 0 ? ws : nullptr, static_cast<int64_t>(need)}},
                       {{mx, n_rows, n_in, size}, operand(mw, size), {mr, n_rows, n_out, size}, ob}));
  if (narrow::fits_fwd(n_rows, n_in, n_out, dtype)) {
    narrow::FwdArgs a{};
    a.x = x, a.w = w, a.b = b, a.res = residual, a.y = y, a.z = z;
    a.xs = x_stride, a.ldw = mw.m.stride, a.ress = residual_stride, a.ys = y_stride, a.zs = z_stride;
    a.rows = static_cast<int32_t>(n_rows), a.n_in = static_cast<int32_t>(n_in), a.n_out = static_cast<int32_t>(n_out);
    a.act = act, a.by_out = mw.by_out;
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, narrow::run_fwd(a, dtype, s));
    return ETPC_OK;
  }
  MatmulArgs a{};
  a.a = x, a.b = w, a.c = y, a.z = z, a.res = residual, a.bias = b;
  a.lda = x_stride, a.ldb = mw.m.stride, a.ldc = y_stride, a.ldz = z_stride, a.ldres = residual_stride;
  a.M = static_cast<int32_t>(n_rows), a.N = static_cast<int32_t>(n_out), a.K = static_cast<int32_t>(n_in);
  a.act = act;
  const MatmulForm form = mw.by_out ? MatmulForm::kRowsCols : MatmulForm::kRowsRows;
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, run_product(a, form, dtype, ws, s));
  return ETPC_OK;
}

etpc_status etpc_linear_workspace_size(int64_t n_rows, int64_t n_in, int64_t n_out, int32_t dtype, size_t* bytes) {
  if (bytes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null output");
  ETPC_TRY(check_layer(n_rows, n_in, n_out, dtype, ETPC_ACT_NONE));
  *bytes = n_rows > 0 ? forward_space(n_rows, n_in, n_out, dtype) : 0;
  return ETPC_OK;
}

etpc_status etpc_linear_backward_workspace_size(int64_t n_rows, int64_t n_in, int64_t n_out, int32_t dtype, int32_t act,
                                                size_t* bytes) {
  if (bytes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null output");
  ETPC_TRY(check_layer(n_rows, n_in, n_out, dtype, act));
  *bytes = n_rows > 0 ? linear_space(n_rows, n_in, n_out, dtype, act).bytes : 0;
  return ETPC_OK;
}

etpc_status etpc_linear_backward(int64_t n_rows, int64_t n_in, int64_t n_out, int32_t dtype, const void* x,
                                 int64_t x_stride, const void* w, int64_t w_in_stride, int64_t w_out_stride,
                                 const void* y_bar, int64_t y_bar_stride, const void* z, int64_t z_stride, int32_t act,
                                 void* x_bar, int64_t x_bar_stride, void* w_bar, int64_t w_bar_in_stride,
                                 int64_t w_bar_out_stride, float* b_bar, void* ws, size_t ws_bytes, hipStream_t s) {
  ETPC_TRY(check_layer(n_rows, n_in, n_out, dtype, act));
  const int64_t size = size_of(dtype);
  Weights mwb{{"w_bar", nullptr, 0}, 0, 0, true};
  if (w_bar != nullptr)
    ETPC_TRY(make_weights("w_bar", w_bar, w_bar_in_stride, w_bar_out_stride, n_in, n_out, dtype, true, &mwb));
  const Operand obb{"b_bar", b_bar, 4 * n_out};
  ETPC_TRY(check_floats({obb}));
  if (n_rows == 0) {
    ETPC_TRY(check_apart({operand(mwb, size), obb}, {}));
    if (w_bar != nullptr)
      ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_sum_parts(nullptr, 0, mwb.rows, mwb.cols, w_bar, mwb.m.stride, nullptr, 0, dtype, s));
    if (b_bar != nullptr) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_fill(b_bar, n_out, 0.f, s));
    return ETPC_OK;
  }
  const Mat mx{"x", x, x_stride}, my{"y_bar", y_bar, y_bar_stride}, mz{"z", z, z_stride},
      mxb{"x_bar", x_bar, x_bar_stride};
  Weights mw{{"w", nullptr, 0}, 0, 0, true};
  if (w_bar != nullptr) ETPC_TRY(check_mat(mx, n_rows, n_in, dtype, false));
  if (x_bar != nullptr) {
    ETPC_TRY(make_weights("w", w, w_in_stride, w_out_stride, n_in, n_out, dtype, false, &mw));
    ETPC_TRY(check_mat(mxb, n_rows, n_in, dtype, true));
  }
  ETPC_TRY(check_mat(my, n_rows, n_out, dtype, false));
  if (act != ETPC_ACT_NONE) ETPC_TRY(check_mat(mz, n_rows, n_out, dtype, false));
  const LinearSpace space = linear_space(n_rows, n_in, n_out, dtype, act);
  const bool any = x_bar != nullptr || w_bar != nullptr || b_bar != nullptr;
  if (any) ETPC_TRY(check_parts(ws, ws_bytes, space.bytes));
  ETPC_TRY(check_apart({{mxb, n_rows, n_in, size}, operand(mwb, size), obb,
                        {"the workspace", any ? ws : nullptr, static_cast<int64_t>(space.bytes)}},
                       {{mx, n_rows, w_bar != nullptr ? n_in : 0, size}, operand(mw, size), {my, n_rows, n_out, size},
                        {mz, n_rows, act != ETPC_ACT_NONE ? n_out : 0, size}}));
  if (!any) return ETPC_OK;

  if (narrow::fits_bwd(n_rows, n_in, n_out, dtype)) {
    narrow::BwdArgs a{};
    const bool sums = w_bar != nullptr || b_bar != nullptr;
    a.x = x, a.w = w, a.y_bar = y_bar, a.z = act != ETPC_ACT_NONE ? z : nullptr, a.x_bar = x_bar;
    if (sums) a.part = static_cast<float*>(ws);
    a.xs = x_stride, a.ldw = mw.m.stride, a.ybs = y_bar_stride, a.zs = z_stride, a.xbs = x_bar_stride;
    a.rows = static_cast<int32_t>(n_rows), a.n_in = static_cast<int32_t>(n_in), a.n_out = static_cast<int32_t>(n_out);
    a.act = act, a.by_out = mw.by_out, a.wb_by_out = mwb.by_out, a.w_sums = w_bar != nullptr;
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, narrow::run_bwd(a, dtype, s));
    if (sums)
      ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_sum_parts(a.part, narrow::bwd_groups(n_rows), mwb.by_out ? n_in : n_out,
                                                       mwb.by_out ? n_out : n_in, w_bar, mwb.m.stride, b_bar, n_out, dtype, s));
    return ETPC_OK;
  }
  char* const at = static_cast<char*>(ws);
  float* const w_part = reinterpret_cast<float*>(at + space.z_bar);
  float* const b_part = reinterpret_cast<float*>(at + space.z_bar + space.w_part);
  void* const x_part = at + space.z_bar + space.w_part + space.b_part;
  const int32_t rows = static_cast<int32_t>(n_rows), in = static_cast<int32_t>(n_in), out = static_cast<int32_t>(n_out);
  const void* z_bar = y_bar;
  int64_t z_bar_stride = y_bar_stride;
  if (act != ETPC_ACT_NONE || b_bar != nullptr) {
    SlopeArgs a{};
    a.y_bar = y_bar, a.ybs = y_bar_stride, a.rows = rows, a.cols = out, a.act = act;
    if (act != ETPC_ACT_NONE) {
      a.z = z, a.zs = z_stride;
      if (x_bar != nullptr || w_bar != nullptr) a.z_bar = at, a.zbs = space.z_bar_stride;
      z_bar = at, z_bar_stride = space.z_bar_stride;
    }
    if (b_bar != nullptr) a.part = b_part;
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_slope(a, dtype, s));
    if (b_bar != nullptr)
      ETPC_LAUNCH(ETPC_KIND_NODEWISE,
                  launch_sum_parts(b_part, slope_parts(rows, out), 1, n_out, b_bar, n_out, nullptr, 0, ETPC_F32, s));
  }
  if (x_bar != nullptr) {
    MatmulArgs a{};
    a.a = z_bar, a.lda = z_bar_stride, a.b = w, a.ldb = mw.m.stride, a.c = x_bar, a.ldc = x_bar_stride;
    a.M = rows, a.N = in, a.K = out;
    const MatmulForm form = mw.by_out ? MatmulForm::kRowsRows : MatmulForm::kRowsCols;
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, run_product(a, form, dtype, x_part, s));
  }
  if (w_bar != nullptr) {
    MatmulArgs a = weight_product(n_rows, n_in, n_out, mwb.by_out);
    a.a = mwb.by_out ? x : z_bar, a.lda = mwb.by_out ? x_stride : z_bar_stride;
    a.b = mwb.by_out ? z_bar : x, a.ldb = mwb.by_out ? z_bar_stride : x_stride;
    a.c = w_bar, a.ldc = mwb.m.stride;
    const MatmulShape shape = matmul_shape(a, MatmulForm::kColsCols, dtype, true);
    if (shape.splits > 1) a.part = w_part;
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_matmul(a, MatmulForm::kColsCols, dtype, shape, s));
    if (shape.splits > 1)
      ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_sum_parts(w_part, shape.splits, a.M, a.N, w_bar, a.ldc, nullptr, 0, dtype, s));
  }
  return ETPC_OK;
}

}  // extern "C"
