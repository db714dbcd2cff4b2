// Launches of the global gradient norm and of clipping (internal).
#pragma once

#include "common.hpp"

namespace etpc {

// How the tensors are cut: pieces of `chunk` elements (each tensor's last one shorter), tables of
// at most kTensors tensors a launch, at most `groups` workgroups a launch, one partial result each.
struct NormPlan {
  int32_t chunk, launches, groups;
  int64_t parts;        // partial results of all launches
};
constexpr int kTensors = 112;   // 3.6 KB of a launch's 4 KB of arguments
NormPlan norm_plan(int32_t n, const int64_t* sizes);

// Partial results (doubles, norm_plan's number of them) of all tensors, then the norm from them.
hipError_t launch_norm_parts(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, bool max,
                             double* parts, hipStream_t s);
hipError_t launch_norm_finish(const double* parts, int64_t count, bool max, float* norm, hipStream_t s);
// Every workgroup takes the norm from the partial results, the first writes it; outs may be the
// gradients themselves.
hipError_t launch_clip(int32_t n, const void* const* grads, void* const* outs, const int64_t* sizes,
                       const int32_t* dtypes, bool max, float max_norm, const double* parts, float* norm, hipStream_t s);

}  // namespace etpc
