// Launches of the global gradient norm and of clipping (internal).
#pragma once

#include "common.hpp"

namespace etpc {

// How the work is cut: tables of at most kTensors tensors a launch; a launch's tensors in units of kUnit
// elements (each tensor's last one shorter), dealt in equal runs to at most `groups` workgroups, one
// partial result each.
struct NormPlan {
  int32_t launches, groups;
  int64_t parts;        // partial results of all launches
};
constexpr int kTensors = 120;   // 3.8 KB of a launch's 4 KB of arguments
constexpr int kUnit = 2048;
NormPlan norm_plan(int32_t n, const int64_t* sizes);

// Partial results (doubles, norm_plan's number of them) of all tensors, then the norm from them.
hipError_t launch_norm_parts(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, bool max,
                             double* parts, hipStream_t s);
hipError_t launch_norm_finish(const double* parts, int64_t count, bool max, float* norm, hipStream_t s);
// Clips by the norm, which is taken from the partial results here and written; outs may be the gradients
// themselves (or null: they are).
hipError_t launch_clip(int32_t n, const void* const* grads, void* const* outs, const int64_t* sizes,
                       const int32_t* dtypes, bool max, float max_norm, const double* parts, float* norm, hipStream_t s);

}  // namespace etpc
