// Division by a number that the host fixes for a launch.
#pragma once

#include <cuda_runtime.h>

namespace nf {

// Division of n < 2^31 by a number fixed for the launch, by a product and a
// shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (hi32(n m) + n) >> s.
struct FastDiv {
  unsigned d, m, s;
  void set(unsigned v) {
    d = v;
    for (s = 0; (1ull << s) < v; ++s) {}
    m = (unsigned)(((1ull << 32) * ((1ull << s) - v)) / v + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((unsigned)n, m) + (unsigned)n) >> s);
  }
};

}  // namespace nf
