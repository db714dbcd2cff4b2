// C ABI of the gradient norm and clipping: argument checks on the host, then their launches.
#include <algorithm>
#include <new>
#include <vector>

#include "grad_norm.hpp"
#include "kernels.hpp"
#include "operands.hpp"
#include "profile.hpp"

namespace etpc {
namespace {

constexpr int64_t kMaxElements = int64_t{1} << 48;

etpc_status check_list(int32_t n, const int64_t* sizes) {
  if (n < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative number of tensors");
  if (n > 0 && sizes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null sizes");
  int64_t total = 0;
  for (int32_t k = 0; k < n; ++k) {
    if (sizes[k] < 0) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "negative size");
    if (sizes[k] > kMaxElements - total) ETPC_FAIL(ETPC_ERR_OVERFLOW, "at most 2^48 elements");
    total += sizes[k];
  }
  return ETPC_OK;
}

etpc_status check_tensors(int32_t n, const void* const* p, const int64_t* sizes, const int32_t* dtypes) {
  if (n > 0 && (p == nullptr || dtypes == nullptr)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null tensor list");
  for (int32_t k = 0; k < n; ++k) {
    if (dtypes[k] != ETPC_F32 && dtypes[k] != ETPC_BF16 && dtypes[k] != ETPC_F16)
      ETPC_FAIL(ETPC_ERR_INVALID_ARG, "bad dtype");
    if (sizes[k] == 0) continue;
    if (p[k] == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null tensor");
    if (reinterpret_cast<uintptr_t>(p[k]) % static_cast<uintptr_t>(size_of(dtypes[k])) != 0)
      ETPC_FAIL(ETPC_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
  }
  return ETPC_OK;
}

etpc_status check_norm(int32_t ord, const float* norm) {
  if (ord != ETPC_NORM_2 && ord != ETPC_NORM_MAX) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "bad norm");
  if (norm == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null norm");
  return check_floats({{"norm", norm, 4}});
}

size_t parts_size(const NormPlan& plan) { return static_cast<size_t>(plan.parts) * sizeof(double); }

etpc_status check_space(const void* ws, size_t have, size_t need) {
  ETPC_TRY(check_parts(ws, have, need));
  if (need > 0 && reinterpret_cast<uintptr_t>(ws) % sizeof(double) != 0)
    ETPC_FAIL(ETPC_ERR_WORKSPACE, "workspace is not aligned to doubles");
  return ETPC_OK;
}

// Memory that a call reads or writes.
struct Extent {
  int64_t at, end;
  bool written;
};
// Whether any written extent meets another one.
bool any_shared(std::vector<Extent>& all) {
  std::sort(all.begin(), all.end(), [](const Extent& a, const Extent& b) { return a.at < b.at; });
  int64_t written = 0, any = 0;   // ends of what starts before
  for (const Extent& e : all) {
    if (e.at < written || (e.written && e.at < any)) return true;
    any = std::max(any, e.end);
    if (e.written) written = std::max(written, e.end);
  }
  return false;
}

etpc_status check_shared(int32_t n, const void* const* grads, const void* const* outs, const int64_t* sizes,
                         const int32_t* dtypes, const float* norm, const void* ws, size_t need) {
  std::vector<Extent> all;
  all.reserve(2 * static_cast<size_t>(n) + 2);
  const auto add = [&](const void* p, int64_t bytes, bool written) {
    const int64_t at = Operand::address(p);
    if (bytes > 0) all.push_back(Extent{at, at + bytes, written});
  };
  for (int32_t k = 0; k < n; ++k) {
    const int64_t bytes = sizes[k] * size_of(dtypes[k]);
    if (outs == nullptr || outs[k] != grads[k]) add(grads[k], bytes, false);
    if (outs != nullptr) add(outs[k], bytes, true);
  }
  add(norm, 4, true);
  add(ws, static_cast<int64_t>(need), true);
  if (any_shared(all)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "written tensors, the norm or the workspace overlap other operands");
  return ETPC_OK;
}

}  // namespace
}  // namespace etpc

using namespace etpc;

extern "C" {

etpc_status etpc_grad_norm_workspace_size(int32_t n, const int64_t* sizes, size_t* bytes) {
  if (bytes == nullptr) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "null output");
  ETPC_TRY(check_list(n, sizes));
  *bytes = parts_size(norm_plan(n, sizes));
  return ETPC_OK;
}

etpc_status etpc_grad_norm(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t ord,
                           float* norm, void* ws, size_t ws_bytes, hipStream_t s) {
  ETPC_TRY(check_list(n, sizes));
  ETPC_TRY(check_norm(ord, norm));
  ETPC_TRY(check_tensors(n, grads, sizes, dtypes));
  const NormPlan plan = norm_plan(n, sizes);
  ETPC_TRY(check_space(ws, ws_bytes, parts_size(plan)));
  try {
    ETPC_TRY(check_shared(n, grads, nullptr, sizes, dtypes, norm, ws, parts_size(plan)));
  } catch (const std::bad_alloc&) {
    ETPC_FAIL(ETPC_ERR_WORKSPACE, "out of host memory");
  }
  double* const parts = static_cast<double*>(ws);
  const bool max = ord == ETPC_NORM_MAX;
  if (plan.parts > 0) ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_norm_parts(n, grads, sizes, dtypes, max, parts, s));
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_norm_finish(parts, plan.parts, max, norm, s));
  return ETPC_OK;
}

etpc_status etpc_clip_grad_norm(int32_t n, const void* const* grads, void* const* outs, const int64_t* sizes,
                                const int32_t* dtypes, int32_t ord, float max_norm, float* norm, void* ws,
                                size_t ws_bytes, hipStream_t s) {
  ETPC_TRY(check_list(n, sizes));
  ETPC_TRY(check_norm(ord, norm));
  if (!(max_norm >= 0.f)) ETPC_FAIL(ETPC_ERR_INVALID_ARG, "max_norm must be >= 0");
  ETPC_TRY(check_tensors(n, grads, sizes, dtypes));
  const void* const* to = outs != nullptr ? const_cast<const void* const*>(outs) : grads;
  if (outs != nullptr) ETPC_TRY(check_tensors(n, to, sizes, dtypes));
  const NormPlan plan = norm_plan(n, sizes);
  ETPC_TRY(check_space(ws, ws_bytes, parts_size(plan)));
  try {
    ETPC_TRY(check_shared(n, grads, to, sizes, dtypes, norm, ws, parts_size(plan)));
  } catch (const std::bad_alloc&) {
    ETPC_FAIL(ETPC_ERR_WORKSPACE, "out of host memory");
  }
  double* const parts = static_cast<double*>(ws);
  const bool max = ord == ETPC_NORM_MAX;
  if (plan.parts == 0) {
    ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_norm_finish(parts, 0, max, norm, s));
    return ETPC_OK;
  }
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_norm_parts(n, grads, sizes, dtypes, max, parts, s));
  ETPC_LAUNCH(ETPC_KIND_NODEWISE, launch_clip(n, grads, outs, sizes, dtypes, max, max_norm, parts, norm, s));
  return ETPC_OK;
}

}  // extern "C"
