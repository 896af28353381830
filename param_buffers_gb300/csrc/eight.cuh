// Eight elements of a row that one thread moves, bf16 or fp32: consecutive ones, as they lie in memory until they are
// wanted, or single ones far apart.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "wide.cuh"

namespace gtp {

// Eight consecutive elements on their own size (16 bytes of bf16, 32 of fp32): one access, and a load in flight holds no
// more registers than bytes.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);  // bf16 -> fp32 is exact
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
};
template <>
struct Eight<float> {
  uint32_t a[8];
  __device__ __forceinline__ void load(const float *p) { load_32b(p, a); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 0;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(a[i]);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(x[i]);
  }
  __device__ __forceinline__ void store(float *p) const { store_32b(p, a); }
};

__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// v as a type holds it.
template <typename T>
__device__ __forceinline__ float rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ float rounded<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// Eight consecutive elements of a vector whose type is known at run time.
__device__ __forceinline__ void load8_of(const void *p, int f32, int64_t i, float (&x)[8]) {
  if (f32) {
    const float4 a = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i)[0],
                 b = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    Eight<__nv_bfloat16> e;
    e.a = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
    e.get(x);
  }
}
// K single elements TX apart of such a vector, those below n: all loads under way together.
template <int TX, int K>
__device__ __forceinline__ void load_apart_of(const void *p, int f32, int i, int n, float (&x)[K]) {
  if (f32) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = i + k * TX < n ? static_cast<const float *>(p)[i + k * TX] : 0.f;
  } else {
    __nv_bfloat16 raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
      raw[k] = i + k * TX < n ? static_cast<const __nv_bfloat16 *>(p)[i + k * TX] : __nv_bfloat16(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = __bfloat162float(raw[k]);
  }
}
__device__ __forceinline__ float load1_of(const void *p, int f32, int64_t i) {
  return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

}  // namespace gtp
