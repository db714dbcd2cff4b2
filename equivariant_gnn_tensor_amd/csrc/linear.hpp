// Launchers of the dense layer (internal).
#pragma once

#include "common.hpp"

namespace etpc {

// C(m, n) = epilogue(sum_k A(m, k) B(k, n)); see matmul.hpp.  Strides in elements.
struct MatmulArgs {
  const void* a;
  const void* b;
  void* c;
  void* z;              // or null: the sum with its bias, before the activation
  const void* res;      // or null
  const float* bias;    // or null
  float* part;          // or null: fp32 sums of `splits` ranges of k go to part[split][M][N] instead
  int64_t lda, ldb, ldc, ldz, ldres;
  int32_t M, N, K;
  int32_t k_split, splits;
  int32_t act;
  int32_t tiles_m, tiles_n;   // filled in by the launch
};
// Which index of A and of B is contiguous.
enum class MatmulForm { kRowsCols, kRowsRows, kColsCols };   // A by rows (k), B by columns (n), ...

struct MatmulShape {
  int tile;        // side of a workgroup's tile
  int grain;       // bytes a lane of the loads straight into LDS (16, 4), or 0: through registers
  int splits, k_split;
  int stages;      // slices in LDS (three: of the 64 x 64 tile of 16 bits)
};
// The shape for a product; `sums`: of rows (a weight gradient).  Operands' addresses and strides do not
// matter to the splits.
MatmulShape matmul_shape(const MatmulArgs& a, MatmulForm form, int dtype, bool sums);
constexpr int kCus = 256;
// Workgroups of a tile of this side that a CU's LDS holds at once.
constexpr int matmul_resident(int tile, int stages) { return 160 * 1024 / (stages * 128 * 2 * tile); }
hipError_t launch_matmul(const MatmulArgs& a, MatmulForm form, int dtype, const MatmulShape& shape, hipStream_t s);
// Up to two rows: C(m, n) with B contiguous along k (`along`) or along n.  launch_matmul takes it.
constexpr int kFewRows = 2;
hipError_t launch_few_rows(const MatmulArgs& a, bool along, int dtype, hipStream_t s);
namespace mm {
hipError_t launch_f32(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s);
hipError_t launch_bf16(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s);
hipError_t launch_f16(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s);
}  // namespace mm

// z_bar = y_bar act'(z) (null: not written), and per part the column sums of it (null: none):
// part[p][cols], p < slope_parts(rows, cols).
struct SlopeArgs {
  const void* y_bar;
  const void* z;        // or null: act is none
  void* z_bar;          // or null
  float* part;          // or null
  int64_t ybs, zs, zbs;
  int32_t rows, cols, act;
};
int slope_parts(int32_t rows, int32_t cols);
hipError_t launch_slope(const SlopeArgs& a, int dtype, hipStream_t s);

// The epilogue of a product over its partial sums a.part[a.splits][M][N].
hipError_t launch_layer_parts(const MatmulArgs& a, int dtype, hipStream_t s);

// out[r ld + c] = sum_{p < parts} part[p][r cols + c], rounded to the dtype once, and tail[i] = the sums
// of the tail_n numbers that follow in each part; in a fixed order.  out, tail: null skips.  No
// parts: zeros.
hipError_t launch_sum_parts(const float* part, int parts, int64_t rows, int64_t cols, void* out, int64_t ld, float* tail,
                            int64_t tail_n, int dtype, hipStream_t s);

}  // namespace etpc
