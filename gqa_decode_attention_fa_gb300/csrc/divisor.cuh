// Division of 32-bit numbers by a divisor that the host knows (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994): a multiplication and two shifts.
#pragma once

#include <stdint.h>

namespace gqa {

struct Divisor {
  uint32_t factor, shift1, shift2;
  void set(uint32_t d) {  // 1 .. 2^31
    int l = 0;
    while ((1ull << l) < d) ++l;
    factor = static_cast<uint32_t>((((1ull << l) - d) << 32) / d + 1);
    shift1 = l > 0 ? 1 : 0;
    shift2 = l > 0 ? l - 1 : 0;
  }
  __host__ __device__ uint32_t divide(uint32_t a) const {
    const uint32_t t = static_cast<uint32_t>((static_cast<uint64_t>(factor) * a) >> 32);
    return (t + ((a - t) >> shift1)) >> shift2;
  }
};

}  // namespace gqa
