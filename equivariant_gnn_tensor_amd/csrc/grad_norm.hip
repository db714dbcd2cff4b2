// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2) or max |g|,  g *= min(1, max_norm / (norm + 1e-6))
//
// Memory bound: the gradients are read once for the norm, and read and written once more to be
// clipped.  Pointers and sizes travel in the launch's arguments (no copy to the device, so the
// calls can be captured), and the tensors are cut into pieces of one size so that large and small
// ones share the chip evenly.  Squares are exact in 64 bits and their sums neither overflow nor
// lose small tensors beside large ones; the conversions and multiply-adds in 64 bits stay hidden
// behind the loads.  A workgroup leaves one partial result; there are few enough (2048, more only
// with thousands of tensors) that every workgroup of the clipping launch adds them all up itself,
// in one order, instead of a launch between.
#include <algorithm>

#include "grad_norm.hpp"
#include "rows.hpp"

namespace etpc {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

struct Table {
  struct Entry {
    const void* p;
    void* out;
    int64_t n;
    int32_t first;      // its first piece among the launch's
    int32_t dtype;
  };
  Entry t[kTensors];
  int32_t n, pieces, chunk;
};
static_assert(sizeof(Table) + 64 <= 4096, "arguments of a launch");

// The tensor a piece belongs to: the last that starts at or before it (empty ones hold none).
__device__ inline int find(const Table& a, int piece) {
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.t[mid].first <= piece) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <class T, class F>
__device__ inline void for_vectors(const T* __restrict__ p, int n, F&& f) {
  int c = 8 * threadIdx.x;
  for (; c + 8 * kThreads * (kUnroll - 1) + 8 <= n; c += 8 * kThreads * kUnroll) {
    float v[kUnroll][8];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) load<8, true>(p, c + i * 8 * kThreads, n, v[i]);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) f(c + i * 8 * kThreads, v[i]);
  }
  for (; c < n; c += 8 * kThreads) {
    float v[8];
    load<8, false>(p, c, n, v);
    f(c, v);
  }
}

// Partial results are combined as the two norms need: sums, or the larger bit pattern of a
// magnitude (an order in which infinity and then NaN are largest).
__device__ inline double join(double a, double b, bool max) {
  return max ? __longlong_as_double(std::max(__double_as_longlong(a), __double_as_longlong(b))) : a + b;
}

// Over the workgroup, in a fixed order; every thread gets it.
__device__ inline double reduce(double v, bool max) {
  __shared__ double lds[kThreads];
  lds[threadIdx.x] = v;
  __syncthreads();
#pragma unroll
  for (int by = kThreads / 2; by > 0; by /= 2) {
    if (static_cast<int>(threadIdx.x) < by) lds[threadIdx.x] = join(lds[threadIdx.x], lds[threadIdx.x + by], max);
    __syncthreads();
  }
  return lds[0];
}

template <class T>
__device__ inline double piece_norm(const T* p, int n, bool max) {
  double s = 0.0;
  if (max) {
    uint32_t m = 0;
    for_vectors(p, n, [&](int, const float (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) m = std::max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    });
    s = fabs(static_cast<double>(__uint_as_float(m)));
  } else {
    double t[4] = {};
    for_vectors(p, n, [&](int, const float (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k & 3] = fma(static_cast<double>(v[k]), static_cast<double>(v[k]), t[k & 3]);
    });
    s = (t[0] + t[1]) + (t[2] + t[3]);
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const Table a, bool max, double* __restrict__ parts) {
  double s = 0.0;
  for (int piece = blockIdx.x; piece < a.pieces; piece += gridDim.x) {
    const Table::Entry& e = a.t[find(a, piece)];
    const int64_t at = static_cast<int64_t>(piece - e.first) * a.chunk;
    const int n = static_cast<int>(std::min<int64_t>(e.n - at, a.chunk));
    const double v = e.dtype == ETPC_F32    ? piece_norm(static_cast<const float*>(e.p) + at, n, max)
                     : e.dtype == ETPC_BF16 ? piece_norm(static_cast<const Bf16*>(e.p) + at, n, max)
                                            : piece_norm(static_cast<const F16*>(e.p) + at, n, max);
    s = join(s, v, max);
  }
  s = reduce(s, max);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__device__ inline double total(const double* __restrict__ parts, int64_t count, bool max) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) s = join(s, parts[i], max);
  s = reduce(s, max);
  return max ? s : sqrt(s);
}

__global__ __launch_bounds__(kThreads) void finish_kernel(const double* __restrict__ parts, int64_t count, bool max,
                                                          float* norm) {
  const double v = total(parts, count, max);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <class T>
__device__ inline void scale_piece(const T* p, T* out, int n, float by) {
  // in place: a thread reads a vector before it writes it, and no other thread's
  for_vectors(p, n, [&](int c, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= by;
    store<8, false>(out, c, n, v);
  });
}

__global__ __launch_bounds__(kThreads) void clip_kernel(const Table a, bool max, float max_norm,
                                                        const double* __restrict__ parts, int64_t count, float* norm) {
  const double v = total(parts, count, max);
  const float rounded = static_cast<float>(v);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = rounded;
  const bool finite = fabsf(rounded) <= 3.4028234e38f;
  const float by = finite ? static_cast<float>(fmin(1.0, static_cast<double>(max_norm) / (v + 1e-6))) : 1.f;
  for (int piece = blockIdx.x; piece < a.pieces; piece += gridDim.x) {
    const Table::Entry& e = a.t[find(a, piece)];
    if (by == 1.f && e.out == e.p) continue;
    const int64_t at = static_cast<int64_t>(piece - e.first) * a.chunk;
    const int n = static_cast<int>(std::min<int64_t>(e.n - at, a.chunk));
    if (e.dtype == ETPC_F32)
      scale_piece(static_cast<const float*>(e.p) + at, static_cast<float*>(e.out) + at, n, by);
    else if (e.dtype == ETPC_BF16)
      scale_piece(static_cast<const Bf16*>(e.p) + at, static_cast<Bf16*>(e.out) + at, n, by);
    else
      scale_piece(static_cast<const F16*>(e.p) + at, static_cast<F16*>(e.out) + at, n, by);
  }
}

// The launches' tables one after another.
template <class F>
hipError_t for_tables(int32_t n, const void* const* grads, void* const* outs, const int64_t* sizes,
                      const int32_t* dtypes, const NormPlan& plan, F&& launch) {
  Table a;
  a.chunk = plan.chunk;
  for (int32_t k = 0; k < n;) {
    a.n = 0;
    int64_t pieces = 0;
    for (; k < n && a.n < kTensors; ++k) {
      if (sizes[k] == 0) continue;
      a.t[a.n++] = Table::Entry{grads[k], outs != nullptr ? outs[k] : const_cast<void*>(grads[k]), sizes[k],
                                static_cast<int32_t>(pieces), dtypes[k]};
      pieces += (sizes[k] + plan.chunk - 1) / plan.chunk;
    }
    if (a.n == 0) break;
    a.pieces = static_cast<int32_t>(pieces);
    const hipError_t e = launch(a, static_cast<unsigned>(std::min<int64_t>(pieces, plan.groups)));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

NormPlan norm_plan(int32_t n, const int64_t* sizes) {
  int64_t total = 0, full = 0;
  for (int32_t k = 0; k < n; ++k) total += sizes[k], full += sizes[k] > 0;
  NormPlan p{};
  p.chunk = 2048;
  while (p.chunk < (1 << 20) && total / p.chunk > 4096) p.chunk *= 2;
  p.launches = static_cast<int32_t>((full + kTensors - 1) / kTensors);
  p.groups = p.launches > 0 ? std::max(64, 2048 / p.launches) : 0;
  int64_t pieces = 0, held = 0;
  for (int32_t k = 0; k < n; ++k) {
    if (sizes[k] == 0) continue;
    pieces += (sizes[k] + p.chunk - 1) / p.chunk;
    if (++held == kTensors) p.parts += std::min<int64_t>(pieces, p.groups), pieces = held = 0;
  }
  p.parts += std::min<int64_t>(pieces, p.groups);
  return p;
}

hipError_t launch_norm_parts(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, bool max,
                             double* parts, hipStream_t s) {
  return for_tables(n, grads, nullptr, sizes, dtypes, norm_plan(n, sizes), [&](const Table& a, unsigned groups) {
    norm_kernel<<<dim3(groups), dim3(kThreads), 0, s>>>(a, max, parts);
    parts += groups;
    return hipGetLastError();
  });
}

hipError_t launch_norm_finish(const double* parts, int64_t count, bool max, float* norm, hipStream_t s) {
  finish_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(parts, count, max, norm);
  return hipGetLastError();
}

hipError_t launch_clip(int32_t n, const void* const* grads, void* const* outs, const int64_t* sizes,
                       const int32_t* dtypes, bool max, float max_norm, const double* parts, float* norm, hipStream_t s) {
  const NormPlan plan = norm_plan(n, sizes);
  return for_tables(n, grads, outs, sizes, dtypes, plan, [&](const Table& a, unsigned groups) {
    clip_kernel<<<dim3(groups), dim3(kThreads), 0, s>>>(a, max, max_norm, parts, plan.parts, norm);
    norm = nullptr;   // the first launch writes it
    return hipGetLastError();
  });
}

}  // namespace etpc
