// Dropout fused with the residual add, and its gradient; the mask is drawn from a counter-based
// generator (philox.cuh) in both directions and never stored.
//
// Page: "Megatron-LM architecture and source guide" (arganzheng.life), §1 (the transformer layer
// whose projection outputs are dropped and added to the residual stream).
//
//   keep(i, j) = r(i, j) >= T,  T = round(65536 p),  r 16 random bits
//   out = residual + (keep ? x * 65536 / (65536 - T) : 0)         dx = keep ? dout * ... : 0
// p is thus taken to the nearest 1/65536 and the scale is that of the probability in use, so the
// mean is kept exactly; 16 bits a draw make eight elements of one generator call, without which the
// calls, not the bytes, would bound the kernel.  A dropped element contributes 0 whatever it holds
// (NaN and Inf included).  Sums in fp32, one rounding.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "device.h"
#include "philox.cuh"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kThreads = 256;

struct DropArgs {
  const void *x, *residual;
  void *out;
  int64_t rows, cols, x_ld, residual_ld, out_ld;
  uint32_t threshold;
  float scale;
  gtp::RngArgs rng;
};

// Eight consecutive elements as fp32, by 16-byte vectors or, up to `n` of them, one by one.
template <bool VEC>
__device__ __forceinline__ void load8(const float *p, int n, float (&x)[8]) {
  if (VEC) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k] : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int n, float (&x)[8]) {
  if (VEC) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);  // bf16 -> fp32 is exact
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? __bfloat162float(p[k]) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(float *p, int n, const float (&x)[8]) {
  if (VEC) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = x[k];
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int n, const float (&x)[8]) {
  if (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = __float2bfloat16_rn(x[k]);
  }
}

// A thread owns one group of eight columns (one generator call) in ROWS rows at a time, whose loads
// are in flight together; blocks are blockDim.x groups wide and step down the rows.
constexpr int kRows = 2;

template <typename TI, typename TO, bool RES, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropArgs a) {
  gtp::ptx::allow_dependents();
  const int64_t g = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t left = a.cols - 8 * g;
  gtp::ptx::wait_prior_grid();
  if (left <= 0) return;
  const int n = VEC ? 8 : int(min(left, int64_t(8)));
  const uint64_t offset = gtp::rng_offset(a.rng);
  const int64_t step = int64_t(gridDim.y) * blockDim.y;
  for (int64_t r0 = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; r0 < a.rows; r0 += kRows * step) {
    float x[kRows][8], res[kRows][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = r0 + i * step;
      if (row < a.rows) {
        load8<VEC>(static_cast<const TI *>(a.x) + row * a.x_ld + 8 * g, n, x[i]);
        if (RES) load8<VEC>(static_cast<const TO *>(a.residual) + row * a.residual_ld + 8 * g, n, res[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = r0 + i * step;
      if (row < a.rows) {
        const uint4 d = gtp::philox(a.rng.k0, a.rng.k1, uint32_t(g) | (gtp::kStreamDropout << 30), uint32_t(row),
                                    uint32_t(offset), uint32_t(offset >> 32));
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t r = k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu;
          y[k] = r >= a.threshold ? x[i][k] * a.scale : 0.f;
          if (RES) y[k] += res[i][k];
        }
        store8<VEC>(static_cast<TO *>(a.out) + row * a.out_ld + 8 * g, n, y);
      }
    }
  }
}

template <typename TI, typename TO, bool RES>
gtp_status launch(const DropArgs &a, bool vec, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const int64_t groups = (a.cols + 7) / 8;
  int tx = 1;
  while (tx < kThreads && tx < groups) tx *= 2;
  const dim3 block(tx, kThreads / tx);
  const int64_t gx = (groups + tx - 1) / tx, want = (a.rows + block.y * kRows - 1) / (block.y * kRows);
  const int64_t fill = (int64_t(dev.sm_count) * 8 + gx - 1) / gx;  // a grid that fills the SMs
  const dim3 grid(unsigned(gx), unsigned(std::max<int64_t>(1, std::min<int64_t>({want, fill, 65535}))));
  return vec ? gtp::launch_overlapped(dropout_kernel<TI, TO, RES, true>, grid, block, 0, st, "dropout", a)
             : gtp::launch_overlapped(dropout_kernel<TI, TO, RES, false>, grid, block, 0, st, "dropout", a);
}

template <typename TI, typename TO>
gtp_status launch(const DropArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  // vectors where every row of every array starts on 16 bytes and holds whole groups
  const auto whole = [&](const void *p, int64_t ld, size_t es) {
    return gtp::aligned16(p) && (a.rows == 1 || ld * int64_t(es) % 16 == 0);
  };
  const bool vec = a.cols % 8 == 0 && whole(a.x, a.x_ld, sizeof(TI)) && whole(a.out, a.out_ld, sizeof(TO)) &&
                   (!a.residual || whole(a.residual, a.residual_ld, sizeof(TO)));
  return a.residual ? launch<TI, TO, true>(a, vec, dev, st) : launch<TI, TO, false>(a, vec, dev, st);
}

constexpr int64_t kMaxDim = int64_t(1) << 30;

gtp_status run(const void *x, gtp_dtype x_dt, int64_t x_ld, const void *residual, int64_t residual_ld, void *out,
               gtp_dtype out_dt, int64_t out_ld, int64_t rows, int64_t cols, float p, const gtp_rng *rng,
               gtp_stream stream) {
  if ((x_dt != GTP_F32 && x_dt != GTP_BF16) || (out_dt != GTP_F32 && out_dt != GTP_BF16))
    return gtp::fail(GTP_E_DTYPE, "dtypes must be F32 or BF16");
  if (rows < 0 || cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (rows > kMaxDim || cols > kMaxDim || rows > (int64_t(1) << 40) / std::max<int64_t>(cols, 1))
    return gtp::fail(GTP_E_SHAPE, "a dimension above 2^30 or more than 2^40 elements");
  if (!(p >= 0.f && p <= 1.f)) return gtp::fail(GTP_E_ARG, "p must be in [0, 1]");
  if (!rng) return gtp::fail(GTP_E_ARG, "null rng");
  if (reinterpret_cast<uintptr_t>(rng->device_offset) & 7u)
    return gtp::fail(GTP_E_ALIGN, "device_offset must be 8-byte aligned");
  const int64_t max_ld = int64_t(1) << 40;
  if (rows > 1 && (x_ld < cols || out_ld < cols || (residual && residual_ld < cols)))
    return gtp::fail(GTP_E_ARG, "a row stride below cols");
  if (x_ld > max_ld || out_ld > max_ld || residual_ld > max_ld) return gtp::fail(GTP_E_SHAPE, "a row stride above 2^40");
  if (rows == 0 || cols == 0) return GTP_OK;
  if (!x || !out) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t xs = x_dt == GTP_F32 ? 4 : 2, os = out_dt == GTP_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) & uintptr_t(xs - 1)) ||
      ((reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(out)) & uintptr_t(os - 1)))
    return gtp::fail(GTP_E_ALIGN, "arrays must be aligned to their elements");
  if (rows == 1) x_ld = residual_ld = out_ld = cols;
  const gtp::ByteRange o = gtp::byte_range(out, ((rows - 1) * out_ld + cols) * os);
  // in place is fine where every element is read and written by one thread: same start, stride, type
  if (gtp::overlap(o, gtp::byte_range(x, ((rows - 1) * x_ld + cols) * xs)) &&
      !(x == out && x_dt == out_dt && x_ld == out_ld))
    return gtp::fail(GTP_E_ARG, "out overlaps the input and is not it");
  if (residual && gtp::overlap(o, gtp::byte_range(residual, ((rows - 1) * residual_ld + cols) * os)) &&
      !(residual == out && residual_ld == out_ld))
    return gtp::fail(GTP_E_ARG, "out overlaps the residual and is not it");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  DropArgs a = {};
  a.x = x, a.residual = residual, a.out = out;
  a.rows = rows, a.cols = cols, a.x_ld = x_ld, a.residual_ld = residual_ld, a.out_ld = out_ld;
  a.threshold = uint32_t(std::lrint(double(p) * 65536.0));
  a.scale = a.threshold < 65536u ? float(65536.0 / double(65536u - a.threshold)) : 0.f;
  a.rng = gtp::rng_args(rng);
  cudaStream_t st = gtp::as_stream(stream);
  if (x_dt == GTP_F32) return out_dt == GTP_F32 ? launch<float, float>(a, dev, st) : launch<float, __nv_bfloat16>(a, dev, st);
  return out_dt == GTP_F32 ? launch<__nv_bfloat16, float>(a, dev, st) : launch<__nv_bfloat16, __nv_bfloat16>(a, dev, st);
}

}  // namespace

extern "C" gtp_status gtp_dropout_add(const void *x, gtp_dtype x_dt, int64_t x_ld, const void *residual,
                                      int64_t residual_ld, void *out, gtp_dtype out_dt, int64_t out_ld, int64_t rows,
                                      int64_t cols, float p, const gtp_rng *rng, gtp_stream stream) {
  gtp::clear_error();
  return run(x, x_dt, x_ld, residual, residual_ld, out, out_dt, out_ld, rows, cols, p, rng, stream);
}

extern "C" gtp_status gtp_dropout_grad(const void *dout, gtp_dtype dout_dt, int64_t dout_ld, void *dx, gtp_dtype dx_dt,
                                       int64_t dx_ld, int64_t rows, int64_t cols, float p, const gtp_rng *rng,
                                       gtp_stream stream) {
  gtp::clear_error();
  return run(dout, dout_dt, dout_ld, nullptr, 0, dx, dx_dt, dx_ld, rows, cols, p, rng, stream);
}
