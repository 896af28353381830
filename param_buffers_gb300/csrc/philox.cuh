// The counter-based random numbers of the dropout and stochastic-rounding kernels.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3",
// SC 2011): ten rounds of two 32 x 32 -> 64 bit products mix a 128-bit counter under a 64-bit
// key into 128 random bits.  A draw is a pure function of (seed, offset, position), so nothing
// random is stored: a mask is drawn again where it is needed again.
//   key     = seed (low word, high word)
//   counter = (group | stream << 30, row, offset low, offset high)
// The streams keep the draws of one (seed, offset) apart: dropout, the rounding of a rowwise
// view and that of a columnwise view (whose rows are the source's columns).
#pragma once
#include <cstdint>

#include "gtp.h"

namespace gtp {

enum : uint32_t { kStreamDropout = 0, kStreamRoundRow = 1, kStreamRoundCol = 2 };

// The rounds' keys are formed on the host: they are the same for every draw of a call, and read from the
// kernel's parameters they cost the rounds nothing.
constexpr int kPhiloxRounds = 10;

struct RngArgs {
  uint32_t keys[kPhiloxRounds][2];
  uint64_t offset;
  const uint64_t *device_offset;
};

inline RngArgs rng_args(const gtp_rng *r) {
  RngArgs a = {};
  if (r) {
    for (int i = 0; i < kPhiloxRounds; ++i) {
      a.keys[i][0] = uint32_t(r->seed) + uint32_t(i) * 0x9E3779B9u;
      a.keys[i][1] = uint32_t(r->seed >> 32) + uint32_t(i) * 0xBB67AE85u;
    }
    a.offset = r->offset;
    a.device_offset = r->device_offset;
  }
  return a;
}

#ifdef __CUDACC__
// The call's offset; the device word (a captured graph's step count) is added when the kernel runs.  It is read, like
// everything that a kernel before this one may have written, by an ordinary load: loads through the read-only path
// need not stay behind the wait for that kernel.
__device__ __forceinline__ uint64_t rng_offset(const RngArgs &r) {
  return r.device_offset ? r.offset + *r.device_offset : r.offset;
}

__device__ __forceinline__ uint4 philox(const RngArgs &r, uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
#pragma unroll
  for (int i = 0; i < kPhiloxRounds; ++i) {
    const uint64_t p = uint64_t(0xD2511F53u) * c0, q = uint64_t(0xCD9E8D57u) * c2;
    c0 = uint32_t(q >> 32) ^ c1 ^ r.keys[i][0];
    c1 = uint32_t(q);
    c2 = uint32_t(p >> 32) ^ c3 ^ r.keys[i][1];
    c3 = uint32_t(p);
  }
  return make_uint4(c0, c1, c2, c3);
}
#endif

}  // namespace gtp
