// Device helpers of the MXFP4 block format: 32 E2M1 elements under one E8M0 scale byte (OCP
// Microscaling Formats).  A block's scale is 2^(byte - 127):
//   nearest     byte = floor(log2 amax) - 2 + 127, 2 being the exponent of E2M1's largest power of
//               two; elements round to nearest, ties to even, and saturate at 6;
//   stochastic  the least power of two with amax <= 6 scale, so that nothing saturates (a clipped
//               element would bias the mean that the rounding keeps); |x| / scale lies between two
//               grid points and goes up with the probability of its distance from the lower one,
//               in steps of 1/256.
// Both clamp at byte 0.  A block holding NaN or Inf gets byte 0xFF (E8M0 NaN) and codes 0.
#pragma once

#include <cuda_fp4.h>

#include <cstdint>

namespace gtp {
namespace mx4 {

constexpr uint32_t kNanScale = 0xFFu;
constexpr uint32_t kInfBits = 0x7F800000u;

// amax_bits: the largest bit pattern of |x| over the block (non-negative floats order like their
// bits, and NaN orders above Inf, so one integer maximum finds both the amax and a bad block).
template <bool STOCH>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  int b = int(amax_bits >> 23) - 2;
  if (STOCH) b += (amax_bits & 0x7FFFFFu) > 0x400000u ? 1 : 0;  // mantissa above 1.5
  return amax_bits >= kInfBits ? kNanScale : uint32_t(max(b, 0));
}

// 1 / scale, or 0 for the NaN byte (whose block's codes are 0).  Bytes reach at most 253.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return byte == kNanScale ? 0.f : __uint_as_float((254u - byte) << 23);
}

// Eight codes of eight values to nearest, the first in the low nibble.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_E2M1,
                                           cudaRoundNearest))
         << (8 * i);
  return w;
}

// One stochastically rounded code.  |x| / scale times 2^-126 is a float whose top bits are the E2M1
// code itself: exponents 1, 2, 3 for [1, 2), [2, 4), [4, 8) and the subnormals for [0, 1), where the
// product keeps 23 fractional bits (round to nearest).  The 22 bits below the code are the fraction
// of the step to the next point, so adding the random byte in their place, centred, carries into
// the code with the right probability.  At most 6 stays at most 6: its fraction is 0.
__device__ __forceinline__ uint32_t encode1_stochastic(float x, float inv, uint32_t r) {
  const float y = fabsf(x * inv) * 0x1p-126f;
  return ((__float_as_uint(y) + (r << 14) + (1u << 13)) >> 22) | ((__float_as_uint(x) >> 28) & 8u);
}

// Eight of them, with the random bytes of r0 (first four) and r1.
__device__ __forceinline__ uint32_t encode8_stochastic(const float (&x)[8], float inv, uint32_t r0, uint32_t r1) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w |= encode1_stochastic(x[i], inv, ((i < 4 ? r0 : r1) >> (8 * (i & 3))) & 0xFFu) << (4 * i);
  return w;
}

}  // namespace mx4
}  // namespace gtp
