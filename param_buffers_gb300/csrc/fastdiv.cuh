// Division by a number fixed on the host: the GEMMs' unit decode, and the elementwise kernels that split an index
// once per item.
#pragma once
#include <cstdint>

namespace gtp {

// Division of 0 <= n < 2^31 by a fixed d >= 1 as one multiply and a shift (the round-up
// method of Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): with l = ceil(log2 d) and m = ceil(2^(31+l) / d) < 2^32,
// floor(n / d) = (n m) >> (31 + l).
struct FastDiv {
  uint32_t m, s;
};

inline FastDiv make_fastdiv(int d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < uint64_t(d)) ++l;
  const uint64_t num = uint64_t(1) << (31 + l);
  return {uint32_t((num + uint64_t(d) - 1) / uint64_t(d)), 31 + l};
}

#ifdef __CUDACC__
__device__ __forceinline__ int fast_div(int n, FastDiv f) {
  return int((uint64_t(uint32_t(n)) * f.m) >> f.s);
}
#endif

}  // namespace gtp
