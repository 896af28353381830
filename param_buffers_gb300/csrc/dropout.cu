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

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// One thread per group of eight columns.
template <typename TI, typename TO, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropArgs a, int64_t groups,
                                                           int64_t total) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const uint64_t offset = gtp::rng_offset(a.rng);
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t row = i / groups, g = i - row * groups;
    const uint4 d = gtp::philox(a.rng.k0, a.rng.k1, uint32_t(g) | (gtp::kStreamDropout << 30), uint32_t(row),
                                uint32_t(offset), uint32_t(offset >> 32));
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
    const TI *x = static_cast<const TI *>(a.x) + row * a.x_ld;
    const TO *res = static_cast<const TO *>(a.residual) + (RES ? row * a.residual_ld : 0);
    TO *out = static_cast<TO *>(a.out) + row * a.out_ld;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t j = 8 * g + k;
      if (j < a.cols) {
        const uint32_t r = (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
        float v = r >= a.threshold ? to_f32(x[j]) * a.scale : 0.f;
        if (RES) v += to_f32(res[j]);
        out[j] = TO(v);
      }
    }
  }
}

template <typename TI, typename TO>
gtp_status launch(const DropArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const int64_t groups = (a.cols + 7) / 8, total = a.rows * groups;
  const int grid = int(std::min<int64_t>((total + kThreads - 1) / kThreads, int64_t(dev.sm_count) * 8));
  if (a.residual) return gtp::launch_overlapped(dropout_kernel<TI, TO, true>, grid, kThreads, 0, st, "dropout_add", a, groups, total);
  return gtp::launch_overlapped(dropout_kernel<TI, TO, false>, grid, kThreads, 0, st, "dropout", a, groups, total);
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
