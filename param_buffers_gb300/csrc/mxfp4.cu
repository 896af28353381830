// MXFP4 quantization: packed E2M1 elements and one E8M0 scale byte per 32, the rowwise view of a
// matrix and the columnwise one (the rowwise view of its transpose, which dgrad and wgrad contract
// over), and the way back.
//
// Page: "Generalized Tensor Parallelism (GTP)" (Megatron-Core developer guide), §1.3 (native
// low-precision weights, rowwise and columnwise views) with the element and scale formats of the
// OCP Microscaling specification; the rules are in mx4_block.cuh.
//
// A view's rows are padded with zeros to whole blocks, and its scale bytes lie in the tiled layout
// (gtp_sf_tile) with their padding written as zero: the products read whole stages of 256
// contraction elements whatever the size, and a stray 0xFF would turn a zero code into NaN.
#include <cuda_bf16.h>

#include <algorithm>

#include "device.h"
#include "mx4_block.cuh"
#include "philox.cuh"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// One thread per block of a view: element k of view row r is src[r * row_stride + k * elem_stride].
template <typename T, bool STOCH>
__global__ void __launch_bounds__(kThreads)
    mx4_view_kernel(const T *__restrict__ src, int64_t row_stride, int64_t elem_stride, int64_t rows, int64_t len,
                    uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int64_t blocks, int64_t words,
                    int64_t total, uint32_t stream, const gtp::RngArgs rng) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const uint64_t offset = STOCH ? gtp::rng_offset(rng) : 0;
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / (4 * words), b = i - r * (4 * words);
    uint32_t byte = 0;
    if (r < rows && b < blocks) {
      float x[4][8];
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const int64_t e = 32 * b + k;
        x[k >> 3][k & 7] = e < len ? to_f32(src[r * row_stride + e * elem_stride]) : 0.f;
        amax = max(amax, __float_as_uint(x[k >> 3][k & 7]) & 0x7FFFFFFFu);
      }
      byte = gtp::mx4::scale_byte<STOCH>(amax);
      const float inv = gtp::mx4::inv_scale(byte);
      uint32_t w[4] = {0, 0, 0, 0};
      if (byte != gtp::mx4::kNanScale) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 d = make_uint4(0, 0, 0, 0);
          if (STOCH)
            d = gtp::philox(rng.k0, rng.k1, uint32_t(2 * b + h) | (stream << 30), uint32_t(r), uint32_t(offset),
                            uint32_t(offset >> 32));
          w[2 * h] = STOCH ? gtp::mx4::encode8_stochastic(x[2 * h], inv, d.x, d.y) : gtp::mx4::encode8(x[2 * h], inv);
          w[2 * h + 1] =
              STOCH ? gtp::mx4::encode8_stochastic(x[2 * h + 1], inv, d.z, d.w) : gtp::mx4::encode8(x[2 * h + 1], inv);
        }
      }
      *reinterpret_cast<uint4 *>(codes + (r * blocks + b) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    scales[((r >> 7) * words + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3)] = uint8_t(byte);
  }
}

// One thread per block of a view, back to values: exact in bf16 and fp32 (one mantissa bit; the
// smallest magnitude, 2^-128, is a bf16 subnormal).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_values_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows, int64_t len,
                      T *__restrict__ out, int64_t blocks, int64_t words, int64_t total) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / blocks, b = i - r * blocks;
    const uint32_t byte = scales[((r >> 7) * words + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3)];
    const float scale = byte == gtp::mx4::kNanScale ? __uint_as_float(0x7FC00000u)
                        : byte == 0                 ? 0x1p-127f
                                                    : __uint_as_float(byte << 23);
    const uint4 v = *reinterpret_cast<const uint4 *>(codes + (r * blocks + b) * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const uint32_t c = (w[k >> 3] >> (4 * (k & 7))) & 15u, m = c & 7u;
      const float mag = m < 4 ? 0.5f * float(m) : m < 6 ? float(m) - 2.f : 2.f * float(m) - 8.f;
      const float y = (c & 8u ? -mag : mag) * scale;
      if (32 * b + k < len) out[r * len + 32 * b + k] = T(y);
    }
  }
}

struct View {
  uint8_t *codes, *scales;
  int64_t rows, len;
  int64_t blocks() const { return (len + 31) / 32; }
  int64_t words() const { return (blocks() + 3) / 4; }
  int64_t code_bytes() const { return rows * blocks() * 16; }
  int64_t scale_bytes() const { return (rows + 127) / 128 * words() * 512; }
};

int grid_for(int64_t threads, int sm_count) {
  return int(std::max<int64_t>(1, std::min<int64_t>((threads + kThreads - 1) / kThreads, int64_t(sm_count) * 8)));
}

template <typename T>
gtp_status launch_view(const T *src, int64_t row_stride, int64_t elem_stride, const View &v, uint32_t stream_id,
                       const gtp_rng *rng, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const int64_t total = (v.rows + 127) / 128 * 128 * v.words() * 4;
  const int grid = grid_for(total, dev.sm_count);
  const gtp::RngArgs a = gtp::rng_args(rng);
  if (rng)
    return gtp::launch_overlapped(mx4_view_kernel<T, true>, grid, kThreads, 0, st, "mxfp4_quantize", src, row_stride,
                                  elem_stride, v.rows, v.len, v.codes, v.scales, v.blocks(), v.words(), total,
                                  stream_id, a);
  return gtp::launch_overlapped(mx4_view_kernel<T, false>, grid, kThreads, 0, st, "mxfp4_quantize", src, row_stride,
                                elem_stride, v.rows, v.len, v.codes, v.scales, v.blocks(), v.words(), total,
                                stream_id, a);
}

template <typename T>
gtp_status launch_views(const void *src, int64_t ld, const View &row, const View &col, const gtp_rng *rng,
                        const gtp::DeviceInfo &dev, cudaStream_t st) {
  auto *s = static_cast<const T *>(src);
  if (row.codes)
    if (gtp_status r = launch_view(s, ld, int64_t(1), row, gtp::kStreamRoundRow, rng, dev, st)) return r;
  if (col.codes)
    if (gtp_status r = launch_view(s, int64_t(1), ld, col, gtp::kStreamRoundCol, rng, dev, st)) return r;
  return GTP_OK;
}

constexpr int64_t kMaxDim = int64_t(1) << 30;

gtp_status check_view(const View &v, const char *name) {
  if ((v.codes != nullptr) != (v.scales != nullptr))
    return gtp::fail(GTP_E_ARG, "%s: codes and scales come together", name);
  if (!gtp::aligned16(v.codes) || !gtp::aligned16(v.scales))
    return gtp::fail(GTP_E_ALIGN, "%s codes and scales must be 16-byte aligned", name);
  return GTP_OK;
}

}  // namespace

extern "C" gtp_status gtp_mxfp4_quantize(const void *src, gtp_dtype src_dt, int64_t rows, int64_t cols, int64_t src_ld,
                                         uint8_t *row_codes, uint8_t *row_scales, uint8_t *col_codes,
                                         uint8_t *col_scales, const gtp_rng *rng, gtp_stream stream) {
  gtp::clear_error();
  if (src_dt != GTP_F32 && src_dt != GTP_BF16) return gtp::fail(GTP_E_DTYPE, "src must be F32 or BF16");
  if (rows < 0 || cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (rows > kMaxDim || cols > kMaxDim) return gtp::fail(GTP_E_SHAPE, "dimension above 2^30");
  if (rows > (int64_t(1) << 40) / std::max<int64_t>(cols, 1)) return gtp::fail(GTP_E_SHAPE, "matrix too large");
  if (src_ld < cols && rows > 1) return gtp::fail(GTP_E_ARG, "src_ld below cols");
  if (src_ld > (int64_t(1) << 40)) return gtp::fail(GTP_E_SHAPE, "src_ld above 2^40");
  if (rng && (reinterpret_cast<uintptr_t>(rng->device_offset) & 7u))
    return gtp::fail(GTP_E_ALIGN, "device_offset must be 8-byte aligned");
  const View row = {row_codes, row_scales, rows, cols}, col = {col_codes, col_scales, cols, rows};
  if (gtp_status s = check_view(row, "rowwise")) return s;
  if (gtp_status s = check_view(col, "columnwise")) return s;
  if (rows == 0 || cols == 0) return GTP_OK;
  if (!row_codes && !col_codes) return gtp::fail(GTP_E_ARG, "no view to write");
  if (!src) return gtp::fail(GTP_E_ARG, "null src");
  const int64_t es = src_dt == GTP_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(src) & uintptr_t(es - 1))
    return gtp::fail(GTP_E_ALIGN, "src must be aligned to its elements");
  const gtp::ByteRange ranges[5] = {gtp::byte_range(src, ((rows - 1) * src_ld + cols) * es),
                                    gtp::byte_range(row_codes, row_codes ? row.code_bytes() : 0),
                                    gtp::byte_range(row_scales, row_scales ? row.scale_bytes() : 0),
                                    gtp::byte_range(col_codes, col_codes ? col.code_bytes() : 0),
                                    gtp::byte_range(col_scales, col_scales ? col.scale_bytes() : 0)};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (gtp::overlap(ranges[i], ranges[j]))
        return gtp::fail(GTP_E_ARG, "an output overlaps the source or another output");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  cudaStream_t st = gtp::as_stream(stream);
  return src_dt == GTP_F32 ? launch_views<float>(src, src_ld, row, col, rng, dev, st)
                           : launch_views<__nv_bfloat16>(src, src_ld, row, col, rng, dev, st);
}

extern "C" gtp_status gtp_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                                           void *out, gtp_dtype out_dt, gtp_stream stream) {
  gtp::clear_error();
  if (out_dt != GTP_F32 && out_dt != GTP_BF16) return gtp::fail(GTP_E_DTYPE, "out must be F32 or BF16");
  if (rows < 0 || cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (rows > kMaxDim || cols > kMaxDim) return gtp::fail(GTP_E_SHAPE, "dimension above 2^30");
  if (rows > (int64_t(1) << 40) / std::max<int64_t>(cols, 1)) return gtp::fail(GTP_E_SHAPE, "matrix too large");
  if (rows == 0 || cols == 0) return GTP_OK;
  if (!codes || !scales || !out) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t es = out_dt == GTP_F32 ? 4 : 2;
  if (!gtp::aligned16(codes) || !gtp::aligned16(scales))
    return gtp::fail(GTP_E_ALIGN, "codes and scales must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(out) & uintptr_t(es - 1))
    return gtp::fail(GTP_E_ALIGN, "out must be aligned to its elements");
  const View v = {const_cast<uint8_t *>(codes), const_cast<uint8_t *>(scales), rows, cols};
  const gtp::ByteRange o = gtp::byte_range(out, rows * cols * es);
  if (gtp::overlap(o, gtp::byte_range(codes, v.code_bytes())) ||
      gtp::overlap(o, gtp::byte_range(scales, v.scale_bytes())))
    return gtp::fail(GTP_E_ARG, "out overlaps the codes or the scales");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  const int64_t total = rows * v.blocks();
  const int grid = grid_for(total, dev.sm_count);
  cudaStream_t st = gtp::as_stream(stream);
  if (out_dt == GTP_F32)
    return gtp::launch_overlapped(mx4_values_kernel<float>, grid, kThreads, 0, st, "mxfp4_dequantize", codes, scales,
                                  rows, cols, static_cast<float *>(out), v.blocks(), v.words(), total);
  return gtp::launch_overlapped(mx4_values_kernel<__nv_bfloat16>, grid, kThreads, 0, st, "mxfp4_dequantize", codes,
                                scales, rows, cols, static_cast<__nv_bfloat16 *>(out), v.blocks(), v.words(), total);
}
