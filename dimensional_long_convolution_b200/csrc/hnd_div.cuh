// hnd_div.cuh -- division by a number fixed at launch.
#pragma once

#include <stdint.h>

namespace hnd {

// n / d = (n mul) >> 32 >> shift for 0 <= n < 2^31, with mul = ceil(2^(31 + s)
// / d) where 2^(s-1) < d <= 2^s (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994).
struct Div {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int quot(int n) const {
    return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
  }
};
inline Div make_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  if (s == 0) return Div{1, 0, 0};
  return Div{d, static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), s - 1};
}

}  // namespace hnd
