// hnd_philox.cuh -- the counter-based generator of the dropout masks:
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011).
//
// Eight elements share a counter and take 16 bits each: a 32-bit lot apiece
// would cost twice the integer work, and at bf16 rates the ten rounds (about
// 60 issue slots a counter) would then bound the streaming kernels instead of
// memory.  A probability is so rounded to a multiple of 2^-16, and the factor
// of the kept elements is that of the rounded probability, which keeps the
// expectation exact.
#pragma once

#include <stdint.h>

#include "hnd_bounds.cuh"

namespace hnd {

__device__ __forceinline__ uint4 philox10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c.x;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

struct DropState {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropState drop_state(const int64_t* rng) {
  const uint64_t seed = static_cast<uint64_t>(*HND_G(rng)), off = static_cast<uint64_t>(*HND_G(rng + 1));
  return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(off),
          static_cast<uint32_t>(off >> 32)};
}

// The lots of elements 8 group .. 8 group + 7.
__device__ __forceinline__ uint4 drop_lots(const DropState& s, uint64_t group) {
  return philox10(make_uint4(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32), s.o0, s.o1), s.k0,
                  s.k1);
}

// Lot j (0..7) of a group.
__device__ __forceinline__ uint32_t drop_lot(const uint4& w, int j) {
  const uint32_t v = j < 4 ? (j < 2 ? w.x : w.y) : (j < 6 ? w.z : w.w);
  return (j & 1) ? v >> 16 : v & 0xFFFFu;
}

}  // namespace hnd
