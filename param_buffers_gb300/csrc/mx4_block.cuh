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

// Two fp32 values in a register pair, multiplied together: half the multiply instructions.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight codes to nearest of eight scaled values (in pairs), the first in the low nibble.
__device__ __forceinline__ uint32_t codes8(const uint64_t (&y)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n\t"
      "mov.b64 {l0, h0}, %1;\n\tmov.b64 {l1, h1}, %2;\n\tmov.b64 {l2, h2}, %3;\n\tmov.b64 {l3, h3}, %4;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, h0, l0;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, h1, l1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, h2, l2;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, h3, l3;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "l"(y[0]), "l"(y[1]), "l"(y[2]), "l"(y[3]));
  return w;
}

// Eight codes rounded towards zero.
__device__ __forceinline__ uint32_t codes8_cut(const uint64_t (&y)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n\t"
      "mov.b64 {l0, h0}, %1;\n\tmov.b64 {l1, h1}, %2;\n\tmov.b64 {l2, h2}, %3;\n\tmov.b64 {l3, h3}, %4;\n\t"
      "cvt.rs.satfinite.e2m1x4.f32 lo, {h1, l1, h0, l0}, %5;\n\tcvt.rs.satfinite.e2m1x4.f32 hi, {h3, l3, h2, l2}, %5;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "l"(y[0]), "l"(y[1]), "l"(y[2]), "l"(y[3]), "r"(0));
  return w;
}

// What codes8_stochastic takes is x / scale times 2^-126, one product of x with 2^(1 - byte).  Above byte 134
// (values of 2^8 and more) that is no bf16; such a block's values are first multiplied by 2^(120 - byte), which takes
// them to 2^-7 of their share of the scale (exact in bf16 down to 2^-119 of it), and then by 2^-119.
__device__ __forceinline__ bool is_far(uint32_t byte) { return byte > 134u && byte != kNanScale; }
__device__ __forceinline__ float near_factor(uint32_t byte) {  // 2^(120 - byte) of a far block, else 1
  return is_far(byte) ? inv_scale(byte) * 0x1p-7f : 1.f;
}
__device__ __forceinline__ float down_factor(uint32_t byte) {
  return is_far(byte) ? 0x1p-119f : inv_scale(byte) * 0x1p-126f;
}

// Eight codes of eight values (in pairs), scaled and times 2^-126, stochastically, with the random bytes of
// r0 (first four) and r1.  Such a value is a float whose bits below the sign are the E2M1 code itself from bit
// 22 up: exponents 1, 2, 3 for [1, 2), [2, 4), [4, 8) and the subnormals for [0, 1), where the product keeps 23
// fractional bits (round to nearest).  The 22 bits below are the fraction of the step to the next point, so adding
// the random byte in their place, centred (byte << 14 | 1 << 13, one byte permute and one
// multiply-add), carries into the code with the right probability; what is left of the fraction is cut off
// by a conversion that rounds stochastically with no random bits.  At most 6 stays at most 6: its
// fraction is 0.
__device__ __forceinline__ uint32_t codes8_stochastic(const uint64_t (&x)[4], uint32_t r0, uint32_t r1) {
  const uint64_t up = pack2(0x1p126f, 0x1p126f);
  uint64_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t = x[i];
    const uint32_t r = i < 2 ? r0 : r1;
    // byte b of r over 0x80: (byte << 8 | 0x80) << 6
    const uint32_t a = __byte_perm(r, 0x80u, (i & 1) ? 0x5524u : 0x5504u);
    const uint32_t b = __byte_perm(r, 0x80u, (i & 1) ? 0x5534u : 0x5514u);
    y[i] = mul2(pack2(__uint_as_float(uint32_t(t) + a * 64u), __uint_as_float(uint32_t(t >> 32) + b * 64u)), up);
  }
  return codes8_cut(y);
}

}  // namespace mx4
}  // namespace gtp
