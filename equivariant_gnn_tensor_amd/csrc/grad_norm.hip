// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum g^2) or max |g|,  g *= min(1, max_norm / (norm + 1e-6))
//
// Memory bound: the gradients are read once for the norm, and read and written once more to be
// clipped (805 MB: the norm of 201 M fp32 139.6 us, 5.8 TB/s, of 403 M bf16 143).  Pointers and sizes travel in the launch's
// arguments (no copy to the device, so the calls can be captured).  The tensors are one long row of units, dealt in equal runs to the
// workgroups: large and small tensors share the chip evenly, and a workgroup looks for its place
// once.  Squares are exact in 64 bits and their sums neither overflow nor lose small tensors beside
// large ones; the conversions and multiply-adds in 64 bits stay hidden behind the loads.  A
// workgroup leaves one partial result.  Up to 1024 of them every workgroup of the clipping launch
// adds up itself, in one order, instead of a launch between; more take that launch.
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
    int64_t first;      // its first unit among the launch's
    int64_t n_dtype;    // elements, and the dtype from bit 56 on
  };
  Entry t[kTensors];
  int64_t units;
  int32_t n;
};
static_assert(sizeof(Table) + 64 <= 4096, "arguments of a launch");

// f(entry, first element, elements) for each tensor's part of this workgroup's run of units.
template <class F>
__device__ inline void for_run(const Table& a, F&& f) {
  const int64_t each = a.units / gridDim.x, more = a.units % gridDim.x, b = blockIdx.x;
  int64_t u = b * each + (b < more ? b : more);
  const int64_t end = u + each + (b < more ? 1 : 0);
  int lo = 0, hi = a.n - 1;   // the last tensor that starts at or before u
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.t[mid].first <= u) lo = mid;
    else hi = mid - 1;
  }
  for (; u < end; ++lo) {
    const Table::Entry& e = a.t[lo];
    const int64_t next = lo + 1 < a.n ? min(a.t[lo + 1].first, end) : end, size = e.n_dtype & ((int64_t{1} << 56) - 1);
    const int64_t from = (u - e.first) * kUnit, to = min(size, (next - e.first) * kUnit);
    f(e, from, to - from);
    u = next;
  }
}

// f(first element, eight numbers) for each vector of a part, zeros past its end.  A thread reads its own
// elements only, and f may write them (p is not __restrict__): clipping works in place, and the neighbours'
// are being written by other waves.
template <class T, class F>
__device__ inline void for_vectors(const T* p, int64_t n, F&& f) {
  int64_t c = 8 * threadIdx.x;
  for (; c + 8 * kThreads * (kUnroll - 1) + 8 <= n; c += 8 * kThreads * kUnroll) {
    float v[kUnroll][8];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) load<8, true>(p + c, i * 8 * kThreads, 8 * kThreads * kUnroll, v[i]);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) f(c + i * 8 * kThreads, v[i]);
  }
  for (; c < n; c += 8 * kThreads) {
    float v[8];
    load_own<8>(p + c, static_cast<int>(min(n - c, int64_t{8})), v);
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
__device__ inline double piece_norm(const T* p, int64_t n, bool max) {
  double s = 0.0;
  if (max) {
    uint32_t m = 0;
    for_vectors(p, n, [&](int64_t, const float (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) m = std::max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    });
    s = fabs(static_cast<double>(__uint_as_float(m)));
  } else {
    double t[4] = {};
    for_vectors(p, n, [&](int64_t, const float (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k & 3] = fma(static_cast<double>(v[k]), static_cast<double>(v[k]), t[k & 3]);
    });
    s = (t[0] + t[1]) + (t[2] + t[3]);
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const Table a, bool max, double* __restrict__ parts) {
  double s = 0.0;
  for_run(a, [&](const Table::Entry& e, int64_t at, int64_t n) {
    const int dtype = static_cast<int>(e.n_dtype >> 56);
    const double v = dtype == ETPC_F32    ? piece_norm(static_cast<const float*>(e.p) + at, n, max)
                     : dtype == ETPC_BF16 ? piece_norm(static_cast<const Bf16*>(e.p) + at, n, max)
                                          : piece_norm(static_cast<const F16*>(e.p) + at, n, max);
    s = join(s, v, max);
  });
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
__device__ inline void scale_piece(const T* p, T* out, int64_t n, float by) {
  // in place: a thread reads a vector before it writes it
  for_vectors(p, n, [&](int64_t c, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= by;
    store<8, false>(out + c, 0, static_cast<int>(min(n - c, int64_t{8})), v);
  });
}

// parts: the norm is taken from them and written by the first workgroup; null: it is in *norm.
__global__ __launch_bounds__(kThreads) void clip_kernel(const Table a, bool max, float max_norm,
                                                        const double* __restrict__ parts, int64_t count, float* norm) {
  float value;
  if (parts != nullptr) {
    value = static_cast<float>(total(parts, count, max));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = value;
  } else {
    value = *norm;
  }
  const bool finite = fabsf(value) <= 3.4028234e38f;
  const float by = finite ? static_cast<float>(fmin(1.0, static_cast<double>(max_norm) / (value + 1e-6))) : 1.f;
  for_run(a, [&](const Table::Entry& e, int64_t at, int64_t n) {
    if (by == 1.f && e.out == e.p) return;
    const int dtype = static_cast<int>(e.n_dtype >> 56);
    if (dtype == ETPC_F32)
      scale_piece(static_cast<const float*>(e.p) + at, static_cast<float*>(e.out) + at, n, by);
    else if (dtype == ETPC_BF16)
      scale_piece(static_cast<const Bf16*>(e.p) + at, static_cast<Bf16*>(e.out) + at, n, by);
    else
      scale_piece(static_cast<const F16*>(e.p) + at, static_cast<F16*>(e.out) + at, n, by);
  });
}

// The launches' tables one after another.
template <class F>
hipError_t for_tables(int32_t n, const void* const* grads, void* const* outs, const int64_t* sizes,
                      const int32_t* dtypes, const NormPlan& plan, F&& launch) {
  Table a;
  for (int32_t k = 0; k < n;) {
    a.n = 0;
    a.units = 0;
    for (; k < n && a.n < kTensors; ++k) {
      if (sizes[k] == 0) continue;
      a.t[a.n++] = Table::Entry{grads[k], outs != nullptr ? outs[k] : const_cast<void*>(grads[k]), a.units,
                                sizes[k] | static_cast<int64_t>(dtypes[k]) << 56};
      a.units += (sizes[k] + kUnit - 1) / kUnit;
    }
    if (a.n == 0) break;
    const hipError_t e = launch(a, static_cast<unsigned>(std::min<int64_t>(a.units, plan.groups)));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

NormPlan norm_plan(int32_t n, const int64_t* sizes) {
  int64_t full = 0;
  for (int32_t k = 0; k < n; ++k) full += sizes[k] > 0;
  NormPlan p{};
  p.launches = static_cast<int32_t>((full + kTensors - 1) / kTensors);
  // 201 M fp32: the norm 139 us with 1024, 140 with 2048, 141 with 4096; 300 tensors of 200000 112, 111
  // and 112
  p.groups = p.launches > 0 ? std::min(2048, std::max(64, 6144 / p.launches)) : 0;
  int64_t units = 0, held = 0;
  for (int32_t k = 0; k < n; ++k) {
    if (sizes[k] == 0) continue;
    units += (sizes[k] + kUnit - 1) / kUnit;
    if (++held == kTensors) p.parts += std::min<int64_t>(units, p.groups), units = held = 0;
  }
  p.parts += std::min<int64_t>(units, p.groups);
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
  if (plan.parts > 1024) {
    const hipError_t e = launch_norm_finish(parts, plan.parts, max, norm, s);
    if (e != hipSuccess) return e;
    parts = nullptr;
  }
  return for_tables(n, grads, outs, sizes, dtypes, plan, [&](const Table& a, unsigned groups) {
    clip_kernel<<<dim3(groups), dim3(kThreads), 0, s>>>(a, max, max_norm, parts, plan.parts, norm);
    return hipGetLastError();
  });
}

}  // namespace etpc
