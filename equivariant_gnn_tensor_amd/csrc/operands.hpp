// Argument checks that the C entry points over rows share: sizes, strides, alignment, operands
// that share memory, workspaces (host code).
#pragma once

#include <cmath>
#include <initializer_list>

#include "common.hpp"

namespace etpc {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxCols = int64_t{1} << 30;

struct Mat {
  const char* name;
  const void* p;
  int64_t stride;
};

inline int64_t size_of(int32_t dtype) { return dtype == ETPC_F32 ? 4 : 2; }

inline etpc_status check_sizes(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 0 || cols < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative size");
  if (dtype != ETPC_F32 && dtype != ETPC_BF16 && dtype != ETPC_F16) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "bad dtype");
  if (rows > kMaxRows) ETPC_FAIL(ETPC_ERR_OVERFLOW, "n_rows must be < 2^31");
  if (cols > kMaxCols) ETPC_FAIL(ETPC_ERR_OVERFLOW, "n_cols must be <= 2^30");
  return ETPC_OK;
}

inline etpc_status check_mat(const Mat& m, int64_t rows, int64_t cols, int32_t dtype, bool output) {
  if (m.p == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string("null ") + m.name);
  if (reinterpret_cast<uintptr_t>(m.p) % static_cast<uintptr_t>(size_of(dtype)) != 0)
    ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string(m.name) + " is not aligned to its elements");
  const bool fits = m.stride >= cols || (!output && m.stride == 0);
  if (rows > 1 && !fits) ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string(m.name) + ": row stride below n_cols");
  if (rows > 1 && m.stride > (int64_t{1} << 60) / rows)
    ETPC_FAIL(ETPC_ERR_OVERFLOW, std::string(m.name) + ": row stride too large");
  return ETPC_OK;
}

// `rows` runs of `run` bytes, `pitch` bytes apart.
struct Runs {
  int64_t at, rows, run, pitch;
};

// An operand for the overlap check: a matrix, or n bytes (parameters, statistics, workspace).
struct Operand {
  const char* name;
  Runs r;
  Operand(const Mat& m, int64_t rows, int64_t cols, int64_t size)
      : name(m.name), r{address(m.p), rows, cols * size, m.stride * size} {
    if (rows == 1 || m.stride == 0) r.rows = 1, r.pitch = 0;
  }
  Operand(const char* what, const void* p, int64_t n) : name(what), r{address(p), 1, n, 0} {}
  static int64_t address(const void* p) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)); }
};

// Whether the single run `one` meets a run of `many`: the first that ends past its start.
inline bool meets(const Runs& one, const Runs& many) {
  const int64_t left = one.at - many.at - many.run;
  const int64_t r = left < 0 ? 0 : left / many.pitch + 1;
  return r < many.rows && many.at + r * many.pitch < one.at + one.run;
}

// Whether two operands share memory (null ones do not).  Extents may cross where runs do not meet: columns of
// wider rows of one pitch, or a single row between the columns of others.
inline bool overlap(const Runs& a, const Runs& b) {
  if (a.at == 0 || b.at == 0 || a.run == 0 || b.run == 0) return false;
  if (a.at + (a.rows - 1) * a.pitch + a.run <= b.at || b.at + (b.rows - 1) * b.pitch + b.run <= a.at) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows == 1) return meets(a, b);
  if (b.rows == 1) return meets(b, a);
  if (a.pitch == b.pitch) {
    const int64_t s = a.pitch, m = ((b.at - a.at) % s + s) % s;
    return m < a.run || s - m < b.run;
  }
  return true;
}

inline etpc_status check_apart(std::initializer_list<Operand> outs, std::initializer_list<Operand> ins) {
  for (const Operand* o = outs.begin(); o != outs.end(); ++o) {
    for (const Operand& i : ins)
      if (overlap(o->r, i.r)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string(o->name) + " and " + i.name + " overlap");
    for (const Operand* q = outs.begin(); q != o; ++q)
      if (overlap(o->r, q->r)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string(o->name) + " and " + q->name + " overlap");
  }
  return ETPC_OK;
}

// fp32 vectors; null ones pass.
inline etpc_status check_floats(std::initializer_list<Operand> vectors) {
  for (const Operand& v : vectors)
    if (v.r.at % static_cast<int64_t>(sizeof(float)) != 0)
      ETPC_FAIL(ETPC_ERR_INVALID_ARG, std::string(v.name) + " is not aligned to its elements");
  return ETPC_OK;
}

inline etpc_status check_eps(float eps) {
  if (!(eps >= 0.f) || !std::isfinite(eps)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return ETPC_OK;
}

inline size_t parts_bytes(int parts, int64_t sums) {
  return parts > 1 ? static_cast<size_t>(parts) * static_cast<size_t>(sums) * sizeof(float) : 0;
}

inline etpc_status check_parts(const void* ws, size_t have, size_t need) {
  if (need > 0 && ws == nullptr) ETPC_FAIL(ETPC_ERR_WORKSPACE, "workspace is null but the call needs one");
  if (have < need) ETPC_FAIL(ETPC_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
  if (need > 0 && reinterpret_cast<uintptr_t>(ws) % sizeof(float) != 0)
    ETPC_FAIL(ETPC_ERR_WORKSPACE, "workspace is not aligned to floats");
  return ETPC_OK;
}

#define ETPC_TRY(call)                      \
  do {                                      \
    const etpc_status _st = (call);         \
    if (_st != ETPC_OK) return _st;         \
  } while (0)

}  // namespace etpc
