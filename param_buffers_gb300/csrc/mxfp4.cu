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
#include <atomic>

#include "device.h"
#include "mx4_block.cuh"
#include "philox.cuh"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kThreads = 256;

// A tile of 128 x 128 source elements makes exactly one 512-byte atom of scale bytes in each view, so
// a block reads its tile once and writes both views: codes in 64-byte runs, scales as one atom each.
//
// Rows: a thread takes 16 consecutive elements of 4 rows (32 apart), two lanes a block of 32.  On the
// way the tile goes to shared memory; then a thread takes 32 rows of two adjacent columns (bf16, one
// 32-bit word a row) or of one column twice (fp32), so a column's block needs no shuffle.  The words
// of a row are rotated by 8 per 32 rows: the four row blocks of a column, which neighbouring lanes
// hold so that they write its 64 bytes together, then lie in different banks.
constexpr int kTile = 128;

template <typename T>
struct Tile {
  static constexpr int PER = 4 / sizeof(T);            // elements of a 32-bit word
  static constexpr int WORDS = kTile / PER;            // words of a tile row
  static constexpr int THREAD_WORDS = 16 / PER;        // words of a thread's 16 elements
  static constexpr int BYTES = kTile * WORDS * 4;
};

template <int N>
__device__ __forceinline__ void load_words(const uint32_t *p, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
}

// The word of up to two elements, element by element, for a ragged or unaligned source.
__device__ __forceinline__ uint32_t word_of(const float *p, int n) { return n > 0 ? __float_as_uint(*p) : 0u; }
__device__ __forceinline__ uint32_t word_of(const __nv_bfloat16 *p, int n) {
  const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
  return (n > 0 ? uint32_t(q[0]) : 0u) | (n > 1 ? uint32_t(q[1]) << 16 : 0u);
}

// The largest magnitude of a word's elements so far: fp32 one 32-bit maximum, bf16 two 16-bit ones.
template <typename T>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t w);
template <>
__device__ __forceinline__ uint32_t max_magnitude<float>(uint32_t m, uint32_t w) {
  return max(m, w & 0x7FFFFFFFu);
}
template <>
__device__ __forceinline__ uint32_t max_magnitude<__nv_bfloat16>(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7FFF7FFFu);
}

__device__ __forceinline__ float low_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// One block of 32 values under `byte` to 16 bytes of codes; view row r, block b (for the draws).
template <bool STOCH, int N>
__device__ __forceinline__ void encode_run(const float (&x)[N], uint32_t byte, uint32_t (&w)[N / 8], uint32_t stream,
                                           uint32_t r, uint32_t first_group, const gtp::RngArgs &rng, uint64_t offset) {
  const float inv = gtp::mx4::inv_scale(byte);
  const uint32_t keep = byte == gtp::mx4::kNanScale ? 0u : 0xFFFFFFFFu;  // a bad block's codes are 0
#pragma unroll
  for (int h = 0; h < N / 16; ++h) {
    uint4 d = make_uint4(0, 0, 0, 0);
    if (STOCH)
      d = gtp::philox(rng.k0, rng.k1, (first_group + h) | (stream << 30), r, uint32_t(offset), uint32_t(offset >> 32));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = x[16 * h + 8 * q + k];
      w[2 * h + q] = keep & (STOCH ? gtp::mx4::encode8_stochastic(v, inv, q ? d.z : d.x, q ? d.w : d.y)
                                   : gtp::mx4::encode8(v, inv));
    }
  }
}

struct ViewArgs {
  uint8_t *codes, *scales;
  int64_t pitch;  // bytes of a row of codes
  int64_t words;  // atoms of a 128-row tile
};

struct TileArgs {
  const void *src;
  int64_t rows, cols, ld;
  int64_t tiles_n;
  ViewArgs row, col;
  int32_t vec;  // rows on 16 bytes
  gtp::RngArgs rng;
};

template <typename T, bool STOCH, bool ROW, bool COL>
__global__ void __launch_bounds__(kThreads) mx4_tile_kernel(const __grid_constant__ TileArgs a) {
  using F = Tile<T>;
  constexpr int TW = F::THREAD_WORDS;
  extern __shared__ __align__(16) uint32_t tile[];  // COL: [128][WORDS]
  __shared__ __align__(16) uint8_t atom[2][512];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const uint64_t offset = STOCH ? gtp::rng_offset(a.rng) : 0;
  const int tid = threadIdx.x;
  const int64_t tm = blockIdx.x / a.tiles_n, tn = blockIdx.x - tm * a.tiles_n;
  const int seg = tid & 7, r32 = tid >> 3;  // this thread's 16 columns, and its row of every 32
  const int64_t c0 = kTile * tn + 16 * seg;
  const int nc = int(max(int64_t(0), min(int64_t(16), a.cols - c0)));  // its columns inside the matrix
  uint32_t w[4][TW];
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int64_t r = kTile * tm + 32 * it + r32;
    const T *p = static_cast<const T *>(a.src) + r * a.ld + c0;
    if (r >= a.rows) {
#pragma unroll
      for (int i = 0; i < TW; ++i) w[it][i] = 0;
    } else if (a.vec && nc == 16) {
      load_words(reinterpret_cast<const uint32_t *>(p), w[it]);
    } else {
#pragma unroll
      for (int i = 0; i < TW; ++i) w[it][i] = word_of(p + F::PER * i, nc - F::PER * i);
    }
  }
  if (COL) {
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      uint32_t *t = tile + (32 * it + r32) * F::WORDS;
#pragma unroll
      for (int i = 0; i < TW / 4; ++i)
        *reinterpret_cast<uint4 *>(t + ((seg * TW + 4 * i + 8 * it) & (F::WORDS - 1))) =
            make_uint4(w[it][4 * i], w[it][4 * i + 1], w[it][4 * i + 2], w[it][4 * i + 3]);
    }
  }
  if (ROW) {
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int64_t r = kTile * tm + 32 * it + r32;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < TW; ++i) m = max_magnitude<T>(m, w[it][i]);
      if (sizeof(T) == 2) m = max(m & 0xFFFFu, m >> 16) << 16;
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      const uint32_t byte = gtp::mx4::scale_byte<STOCH>(m);
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        x[k] = sizeof(T) == 4 ? __uint_as_float(w[it][k % TW])
                              : (k & 1 ? high_f32(w[it][k >> 1]) : low_f32(w[it][k >> 1]));
      uint32_t codes[2];
      encode_run<STOCH>(x, byte, codes, gtp::kStreamRoundRow, uint32_t(r), uint32_t(8 * tn + seg), a.rng, offset);
      const bool in = r < a.rows && c0 < 2 * a.row.pitch;  // the block exists (two codes a byte)
      if (in) *reinterpret_cast<uint2 *>(a.row.codes + r * a.row.pitch + c0 / 2) = make_uint2(codes[0], codes[1]);
      if ((seg & 1) == 0) atom[0][16 * r32 + 4 * it + (seg >> 1)] = uint8_t(byte);
    }
  }
  __syncthreads();
  if (COL) {
    // lanes 4 p + rb: column pair (bf16) or column (fp32) p of the warp's eight, row block rb
    const int rb = tid & 3;
#pragma unroll
    for (int u = 0; u < 2 / F::PER; ++u) {
      const int p = (tid >> 2) + 64 * u;  // word of the tile row
      const uint32_t *t = tile + 32 * rb * F::WORDS + ((p + 8 * rb) & (F::WORDS - 1));
      uint32_t v[32], m = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        v[k] = t[k * F::WORDS];
        m = max_magnitude<T>(m, v[k]);
      }
#pragma unroll
      for (int e = 0; e < F::PER; ++e) {
        const int c = F::PER * p + e;
        const int64_t gc = kTile * tn + c;
        const uint32_t byte = gtp::mx4::scale_byte<STOCH>(F::PER == 1 ? m : e ? m & 0xFFFF0000u : m << 16);
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = F::PER == 1 ? __uint_as_float(v[k]) : e ? high_f32(v[k]) : low_f32(v[k]);
        uint32_t codes[4];
        encode_run<STOCH>(x, byte, codes, gtp::kStreamRoundCol, uint32_t(gc), uint32_t(8 * tm + 2 * rb), a.rng, offset);
        const int64_t b = 4 * tm + rb;
        if (gc < a.cols && 16 * b < a.col.pitch)
          *reinterpret_cast<uint4 *>(a.col.codes + gc * a.col.pitch + 16 * b) =
              make_uint4(codes[0], codes[1], codes[2], codes[3]);
        atom[1][16 * (c & 31) + 4 * (c >> 5) + rb] = uint8_t(byte);
      }
    }
    __syncthreads();
  }
  // the atoms whole: rows, columns and blocks outside the matrix hold zeros, whose byte is 0
  if (ROW && tid < 32)
    reinterpret_cast<uint4 *>(a.row.scales + (tm * a.row.words + tn) * 512)[tid] = reinterpret_cast<uint4 *>(atom[0])[tid];
  if (COL && tid >= 32 && tid < 64)
    reinterpret_cast<uint4 *>(a.col.scales + (tn * a.col.words + tm) * 512)[tid - 32] =
        reinterpret_cast<uint4 *>(atom[1])[tid - 32];
}

// Eight values a thread, back from a view: exact in bf16 and fp32 below 2^128 (one mantissa bit; the
// smallest magnitude, 2^-128, is a bf16 subnormal).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    mx4_values_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows, int64_t len,
                      T *__restrict__ out, int64_t blocks, int64_t words) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int64_t g = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, b = g >> 2;
  const int64_t left = len - 8 * g;
  if (left <= 0) return;
  const uint8_t *sf = scales + (b >> 2) * 512 + (b & 3);
  for (int64_t r = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; r < rows; r += int64_t(gridDim.y) * blockDim.y) {
    const uint32_t byte = __ldg(sf + (r >> 7) * words * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4);
    const float scale = byte == gtp::mx4::kNanScale ? __uint_as_float(0x7FC00000u)
                        : byte == 0                 ? 0x1p-127f
                                                    : __uint_as_float(byte << 23);
    const uint32_t w = __ldcs(reinterpret_cast<const uint32_t *>(codes + r * blocks * 16) + g);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t((w >> (8 * i)) & 0xFFu), __NV_E2M1);
      const float2 f = __half22float2(__half2(h));
      x[2 * i] = f.x * scale;
      x[2 * i + 1] = f.y * scale;
    }
    T *o = out + r * len + 8 * g;
    if constexpr (VEC && sizeof(T) == 4) {
      __stcs(reinterpret_cast<float4 *>(o), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4 *>(o) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else if constexpr (VEC) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t *>(&p);
      }
      __stcs(reinterpret_cast<uint4 *>(o), make_uint4(v[0], v[1], v[2], v[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) o[k] = T(x[k]);
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

template <typename T, bool STOCH, bool ROW, bool COL>
gtp_status launch_tiles(const TileArgs &a, int64_t tiles, const gtp::DeviceInfo &dev, cudaStream_t st) {
  constexpr int smem = COL ? Tile<T>::BYTES : 0;
  constexpr auto kernel = mx4_tile_kernel<T, STOCH, ROW, COL>;
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> configured{0};
    const uint64_t bit = uint64_t(1) << (dev.device & 63);
    if (!(configured.load() & bit)) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      configured.fetch_or(bit);
    }
  }
  return gtp::launch_overlapped(kernel, dim3(unsigned(tiles)), kThreads, smem, st, "mxfp4_quantize", a);
}

template <typename T, bool STOCH>
gtp_status launch_views(const TileArgs &a, int64_t tiles, const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (!a.col.codes) return launch_tiles<T, STOCH, true, false>(a, tiles, dev, st);
  if (!a.row.codes) return launch_tiles<T, STOCH, false, true>(a, tiles, dev, st);
  return launch_tiles<T, STOCH, true, true>(a, tiles, dev, st);
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
  TileArgs a = {};
  a.src = src;
  a.rows = rows, a.cols = cols, a.ld = rows > 1 ? src_ld : 0;
  a.tiles_n = (cols + kTile - 1) / kTile;
  a.row = {row_codes, row_scales, row.blocks() * 16, row.words()};
  a.col = {col_codes, col_scales, col.blocks() * 16, col.words()};
  a.vec = gtp::aligned16(src) && a.ld * es % 16 == 0;
  a.rng = gtp::rng_args(rng);
  const int64_t tiles = (rows + kTile - 1) / kTile * a.tiles_n;
  if (tiles > INT32_MAX) return gtp::fail(GTP_E_SHAPE, "more than 2^31 - 1 tiles of 128 x 128");
  if (src_dt == GTP_F32) return rng ? launch_views<float, true>(a, tiles, dev, st) : launch_views<float, false>(a, tiles, dev, st);
  return rng ? launch_views<__nv_bfloat16, true>(a, tiles, dev, st) : launch_views<__nv_bfloat16, false>(a, tiles, dev, st);
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
  cudaStream_t st = gtp::as_stream(stream);
  const int64_t groups = (cols + 7) / 8;
  int tx = 4;  // a block's four words of codes side by side
  while (tx < kThreads && tx < groups) tx *= 2;
  const dim3 block(tx, kThreads / tx);
  const int64_t gx = (groups + tx - 1) / tx, want = (rows + block.y - 1) / block.y;
  const int64_t fill = (int64_t(dev.sm_count) * 16 + gx - 1) / gx;
  const dim3 grid(unsigned(gx), unsigned(std::max<int64_t>(1, std::min<int64_t>({want, fill, 65535}))));
  const bool vec = cols % 8 == 0 && gtp::aligned16(out);
  const auto go = [&](auto *kernel, auto *o) {
    return gtp::launch_overlapped(kernel, grid, block, 0, st, "mxfp4_dequantize", codes, scales, rows, cols, o,
                                  v.blocks(), v.words());
  };
  if (out_dt == GTP_F32)
    return vec ? go(mx4_values_kernel<float, true>, static_cast<float *>(out))
               : go(mx4_values_kernel<float, false>, static_cast<float *>(out));
  return vec ? go(mx4_values_kernel<__nv_bfloat16, true>, static_cast<__nv_bfloat16 *>(out))
             : go(mx4_values_kernel<__nv_bfloat16, false>, static_cast<__nv_bfloat16 *>(out));
}
