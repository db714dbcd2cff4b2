// Counter-based dropout masks: Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011), eight 16-bit fields per call.
#pragma once

#include "common.hpp"

namespace etpc {

// Dropout of a call as the kernels see it: drop where a field < threshold, multiply the
// rest by scale.  threshold == 0 means no dropout at all.
struct DropArgs {
  uint32_t threshold;          // rint(65536 p), 0..65536
  float scale;                 // 65536 / (65536 - threshold), 0 when everything is dropped
  uint64_t seed;
  uint64_t offset;
  const uint64_t* offset_add;  // [device] added to offset, or null
};

__device__ inline uint64_t drop_offset(const DropArgs& d) {
  return d.offset + (d.offset_add != nullptr ? *d.offset_add : 0);
}

// a ^ b ^ c as one instruction (the truth table of a three-input xor); left to itself the
// compiler takes two, and 16-bit rows spend as long on the generator as on memory (50000 x
// 577 bf16 26.5 us -> 24.9; fp32 rows, memory bound, 48.9 -> 50.3).
__device__ inline uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// The four output words at counter (c0, c1, offset) under key seed.  Ten rounds of two
// 32 x 32 -> 64 bit products each.
struct Philox {
  uint32_t w[4];
};
__device__ inline Philox philox(uint32_t c0, uint32_t c1, uint64_t offset, uint64_t seed) {
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = xor3(static_cast<uint32_t>(p1 >> 32), c1, k0);
    c1 = static_cast<uint32_t>(p1);
    c2 = xor3(static_cast<uint32_t>(p0 >> 32), c3, k1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Philox{{c0, c1, c2, c3}};
}

// v[k] <- kept ? v[k] * scale : 0 for the eight channels of counter (group, row).  A
// dropped value is replaced, not multiplied, so an infinity or NaN there leaves no trace.
__device__ inline void drop8(float (&v)[8], const Philox& r, uint32_t threshold, float scale) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t field = (k & 1) ? r.w[k >> 1] >> 16 : r.w[k >> 1] & 0xFFFFu;
    v[k] = field >= threshold ? v[k] * scale : 0.f;
  }
}

}  // namespace etpc
