// Root-mean-square norm with the residual's addition, its output in bf16 or fp32 and / or as the MXFP8 views that a
// linear's products read; and the values of such views.  The gradient is rmsnorm_grad.cu's.
//
// Pages: "Megatron-LM architecture and source guide" (arganzheng.life), §1 (the transformer layer: a norm before the
// attention block and before the MLP, each on the residual stream); "Generalized Tensor Parallelism (GTP)"
// (Megatron-Core developer guide), §1.3 (MXFP8 rowwise and columnwise views).
//
//   s = x + residual (rounded to the stream's type; s = x without one)     r = 1 / sqrt(mean s^2 + eps) per row
//   y = (s r) w                                                             views: MXFP8 of the fp32 y, one rounding
// Sums in fp32.  One pass over the bytes, a row's elements staying in registers between the sum of squares and the outputs:
// long calls on whole vectors are bound by the bytes, the others by latency as their kernels say.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "device.h"
#include "eight.cuh"
#include "mx_block.cuh"
#include "norm_args.h"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

namespace cg = cooperative_groups;

// Scale byte (row r, block j) of a [rows, blocks] array, at its place in the tiled layout where words (the row's 32-bit
// words there) is not 0.
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t j, int64_t blocks, int64_t words) {
  if (words == 0) return r * blocks + j;
  return ((r >> 7) * words + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

constexpr int kRowThreads = 512;  // of a row, at most
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxCols = 32 * kRowThreads;

struct NormArgs {
  const void *x, *residual, *weight;
  void *sum, *y;
  float *rstd;
  uint8_t *row_codes, *row_scales, *col_codes, *col_scales;
  int64_t rows, cols, x_ld, residual_ld, sum_ld, y_ld;
  int64_t row_words, col_words;  // 0: scales in [rows, blocks] order
  float eps, inv_cols;
  float least;  // sums of squares below it lose bits that matter
  int weight_f32, y_f32, codes_on_32;  // the last: col_codes starts on 32 bytes
};

using gtp::Eight;
using gtp::warp_sum;

// 1 / sqrt(mean + eps) of a row's sum of squares.
__device__ __forceinline__ float rstd_of(const NormArgs &a, float squares) { return rsqrtf(fmaf(squares, a.inv_cols, a.eps)); }

// A row whose squares leave fp32's range, or are so small that they lose bits (NormArgs::least), has them summed again with
// its elements multiplied by a power of two: 2^-72 brings the largest sum of 16384, below 2^270, under 2^126, and one above
// 2^100 has its large terms at 2^-58 and more; 2^100 brings a sum below 2^-100 under 2^100, and the smallest number's square
// to 2^-98.  Rows with NaN or Inf, and rows of zeros, end as without it.
__device__ __forceinline__ bool in_range(const NormArgs &a, float squares) { return (squares >= a.least) & (squares <= 0x1p100f); }
__device__ __forceinline__ float factor_of(float squares) { return squares < 1.f ? 0x1p100f : 0x1p-72f; }
__device__ __forceinline__ float rstd_of(const NormArgs &a, float squares, float factor) {
  return factor * rsqrtf(fmaf(squares, a.inv_cols, a.eps * factor * factor));
}

__device__ __forceinline__ void store_y(const NormArgs &a, int64_t row, int64_t c, const float (&y)[8]) {
  if (a.y_f32) {
    Eight<float> e;
    e.set(y);
    e.store(static_cast<float *>(a.y) + row * a.y_ld + c);
  } else {
    Eight<__nv_bfloat16> e;
    e.set(y);
    e.store(static_cast<__nv_bfloat16 *>(a.y) + row * a.y_ld + c);
  }
}

// A block's scale byte and the factor of its elements, from the largest |y| pattern: the amax, and above every finite
// one's where there is NaN or Inf.  There the factor is NaN and makes every code the format's NaN.
__device__ __forceinline__ uint32_t block_scale(uint32_t bits, float &inv) {
  const uint32_t byte = bits < 0x7F800000u ? gtp::mx::scale_byte(__uint_as_float(bits)) : gtp::mx::kNanScale;
  inv = bits < 0x7F800000u ? gtp::mx::inv_scale(byte) : __uint_as_float(0x7FC00000u);
  return byte;
}

// The rowwise view of eight consecutive elements of a row, `bits` their largest pattern: four lanes hold a block.  All 32
// lanes take part; live: this one's elements exist (whole blocks do or do not).
__device__ __forceinline__ void store_row_view(const NormArgs &a, int64_t row, int64_t c, bool live, const float (&y)[8],
                                               uint32_t bits) {
  bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
  bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 2));
  if (!live) return;
  float inv;
  const uint32_t byte = block_scale(bits, inv);
  *reinterpret_cast<uint2 *>(a.row_codes + row * a.cols + c) =
      make_uint2(gtp::mx::encode4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                 gtp::mx::encode4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
  if ((c & 31) == 0) a.row_scales[scale_at(row, c >> 5, a.cols >> 5, a.row_words)] = uint8_t(byte);
}

// --------------------------------------------------------------------------- forward, row by row

// Sums of N rows at a time over the blockDim.x threads of a row (whole warps; blockDim.y rows a block side by side where
// one warp is a row's).  part: two arrays in turn, so that one barrier each time does.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (&part)[2][N][32], int flip) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = warp_sum(s[i]);
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[flip][i][threadIdx.x >> 5] = s[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = warp_sum(lane < warps ? part[flip][i][lane] : 0.f);
}

// A row that is not in range, once more from memory and at its own scale, by its threads: rstd and what goes by rows.  s:
// what its squares are formed of, the sum or x.  Rows that are clearly in range (or NaN) are left as they are where `known`
// is not set: sums in another order than the kernels', so one next to the border may be formed again, no less exactly.
__device__ __forceinline__ void redo_row(const NormArgs &a, int64_t row, const void *s, int s_f32, int64_t ld, bool known) {
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, tx = blockDim.x;
  float factor = 1.f, squares = 0.f;
  for (int again = 0; again < 2; ++again) {
    float sum = 0.f;
    for (int c = threadIdx.x; c < int(a.cols); c += tx) {
      const float x = gtp::load1_of(s, s_f32, row * ld + c) * factor;
      sum = fmaf(x, x, sum);
    }
    squares = warp_sum(sum);
    if (warps > 1) {
      __syncthreads();
      if (lane == 0) part[threadIdx.x >> 5] = squares;
      __syncthreads();
      squares = warp_sum(lane < warps ? part[lane] : 0.f);
    }
    if (again) break;
    if (!known && !(squares > 0x1p99f) && !(squares < 2.f * a.least)) return;
    factor = factor_of(squares);
  }
  const float r = rstd_of(a, squares, factor);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
  for (int c0 = 0; c0 < int(a.cols); c0 += tx) {
    const int c = c0 + threadIdx.x;
    const bool live = c < int(a.cols);
    const float y = live ? gtp::load1_of(s, s_f32, row * ld + c) * r * gtp::load1_of(a.weight, a.weight_f32, c) : 0.f;
    if (a.y && live) {
      if (a.y_f32) static_cast<float *>(a.y)[row * a.y_ld + c] = y;
      else static_cast<__nv_bfloat16 *>(a.y)[row * a.y_ld + c] = __float2bfloat16_rn(y);
    }
    if (a.row_codes) {  // a warp's 32 columns are a block
      float inv;
      const uint32_t byte = block_scale(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(y) & 0x7FFFFFFFu), inv);
      if (live) a.row_codes[row * a.cols + c] = uint8_t(gtp::mx::encode4(y * inv, 0.f, 0.f, 0.f));
      if (live && lane == 0) a.row_scales[scale_at(row, c >> 5, a.cols >> 5, a.row_words)] = uint8_t(byte);
    }
  }
}

// Calls, so that the kernels keep no registers for them: of one row in the middle, where y may have x's place, and of all
// rows of a block (a warp, where it has rows of its own) at the end ([8192, 4096] bf16 with a residual 42.6 us; checked in the
// middle 45.4, formed there in line 56).
__device__ __noinline__ void redo_one(const NormArgs &a, int64_t row, const void *s, int s_f32, int64_t ld) {
  redo_row(a, row, s, s_f32, ld, true);
}
__device__ __noinline__ void redo_all(const NormArgs &a, const void *s, int s_f32, int64_t ld) {
  if (blockDim.x > 32) __syncthreads();  // every thread's part of the sum is stored
  else __syncwarp();
  for (int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows; row += int64_t(gridDim.x) * blockDim.y)
    redo_row(a, row, s, s_f32, ld, false);
}

// V groups of eight consecutive elements a thread and row, N rows a time: their loads are in flight together and they
// share a barrier.
template <typename TX, typename TS, bool RES, int V, int N>
__global__ void __launch_bounds__(kRowThreads) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][N][32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int tx = blockDim.x;
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  int flip = 0;
  bool fine = true;  // with a residual: all rows are in range
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < a.rows; r0 += N * step, flip ^= 1) {
    Eight<TX> x[N][V];
    Eight<TS> h[N][V];  // the residual, then the sum
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step + threadIdx.y;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (int64_t(v) * tx + threadIdx.x);
        x[i][v].clear();
        h[i][v].clear();
        if (row < a.rows && c < a.cols) {
          x[i][v].load(static_cast<const TX *>(a.x) + row * a.x_ld + c);
          if (RES) h[i][v].load(static_cast<const TS *>(a.residual) + row * a.residual_ld + c);
        }
      }
    }
    float squares[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step + threadIdx.y;
      squares[i] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * (int64_t(v) * tx + threadIdx.x);
        float s[8];
        x[i][v].get(s);
        if (RES) {
          float res[8];
          h[i][v].get(res);
#pragma unroll
          for (int k = 0; k < 8; ++k) s[k] += res[k];
          h[i][v].set(s);  // rounded to the stream's type
          h[i][v].get(s);
          if (row < a.rows && c < a.cols) h[i][v].store(static_cast<TS *>(a.sum) + row * a.sum_ld + c);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) squares[i] = fmaf(s[k], s[k], squares[i]);
      }
    }
    row_sums<N>(squares, part, flip);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = 8 * (int64_t(v) * tx + threadIdx.x);
      const bool live = c < a.cols;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 0.f;
      if (live) gtp::load8_of(a.weight, a.weight_f32, c, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t row = r0 + i * step + threadIdx.y;
        const float r = rstd_of(a, squares[i]);
        if (a.rstd && v == 0 && threadIdx.x == 0 && row < a.rows) a.rstd[row] = r;
        float y[8];
        if (RES) h[i][v].get(y);
        else x[i][v].get(y);
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          y[k] = y[k] * r * w[k];
          bits = max(bits, __float_as_uint(y[k]) & 0x7FFFFFFFu);
        }
        const bool there = RES ? live && row < a.rows : live & (row < a.rows) & in_range(a, squares[i]);
        if (RES && v == 0) fine = fine & in_range(a, squares[i]);
        if (a.y && there) store_y(a, row, c, y);
        if (a.row_codes) store_row_view(a, row, c, there, y, bits);
      }
    }
    if constexpr (!RES) {  // y may be x
      bool now = true;
#pragma unroll
      for (int i = 0; i < N; ++i) now = now & in_range(a, squares[i]);
      if (!now) {
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          float sq = squares[0];
#pragma unroll
          for (int q = 1; q < N; ++q) sq = i == q ? squares[q] : sq;
          const int64_t row = r0 + i * step + threadIdx.y;
          if (!in_range(a, sq) && row < a.rows) redo_one(a, row, a.x, sizeof(TX) == 4, a.x_ld);
        }
      }
    }
  }
  if (RES && !fine) redo_all(a, a.sum, sizeof(TS) == 4, a.sum_ld);
}

// Rows that start anywhere: the elements TX apart are a thread's, so that a warp's accesses stand side by side whatever a
// row's alignment.  One row a block of TX threads, K elements a thread, or (TX 32) eight rows.  [8001, 1535] bf16 onto an
// fp32 stream 28.3 us (5.2 TB/s): bound by the single accesses' latency and count.
template <typename T, typename TS, bool RES, int TX, int K>
__global__ void __launch_bounds__(TX == 32 ? 256 : TX, K == 16 ? 1024 / TX : RES && TX == 256 ? 5 : 0) norm_elements_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][1][32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int cols = int(a.cols), t = threadIdx.x;
  int flip = 0;
  bool fine = true;
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < a.rows; r0 += int64_t(gridDim.x) * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < a.rows;
    const T *const x = static_cast<const T *>(a.x) + row * a.x_ld + t;
    const TS *const res = static_cast<const TS *>(a.residual) + (RES ? row * a.residual_ld + t : 0);
    TS *const sum = static_cast<TS *>(a.sum) + (RES ? row * a.sum_ld + t : 0);
    float h[K], squares[1] = {0.f};
    T in[K];
    TS old[RES ? K : 1];  // all loads, as they lie in memory, before the first store
#pragma unroll
    for (int k = 0; k < K; ++k) {
      in[k] = live && t + k * TX < cols ? x[k * TX] : T(0.f);
      if (RES) old[RES ? k : 0] = live && t + k * TX < cols ? res[k * TX] : TS(0.f);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = float(in[k]);
    if (RES) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        h[k] = gtp::rounded<TS>(h[k] + float(old[RES ? k : 0]));
        if (live && t + k * TX < cols) gtp::store1(sum + k * TX, h[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) squares[0] = fmaf(h[k], h[k], squares[0]);
    row_sums<1>(squares, part, flip);
    const float r = rstd_of(a, squares[0]);
    if (!RES && !in_range(a, squares[0])) {
      if (live) redo_row(a, row, a.x, sizeof(T) == 4, a.x_ld, true);
      continue;
    }
    if (RES) fine = fine & in_range(a, squares[0]);
    if (a.rstd && live && t == 0) a.rstd[row] = r;
    if (!a.y || !live) continue;
    const int64_t at = row * a.y_ld + t;
    float w[K];
    if constexpr (RES) {  // one after the other, in the shadow of the sum's stores: 28.3 us of the case above, together 29.2
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = t + k * TX < cols ? gtp::load1_of(a.weight, a.weight_f32, t + k * TX) : 0.f;
    } else {  // all together: [8192, 8001] bf16 88 us, one after the other 93
      gtp::load_apart_of<TX>(a.weight, a.weight_f32, t, cols, w);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t + k * TX < cols) {
        const float y = h[k] * r * w[k];
        if (a.y_f32) static_cast<float *>(a.y)[at + k * TX] = y;
        else static_cast<__nv_bfloat16 *>(a.y)[at + k * TX] = __float2bfloat16_rn(y);
      }
  }
  if (RES && !fine) redo_all(a, a.sum, sizeof(TS) == 4, a.sum_ld);
}

// --------------------------------------------------------------------------- forward with the columnwise view

// The sums of squares of a warp's four rows, lane 8 i + b with block b's part of row i; added up in the same order in every
// block and lane.
__device__ __forceinline__ float row_squares(const float (&squares)[32][8], int blocks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float t = (lane & 7) < blocks ? squares[4 * warp + (lane >> 3)][lane & 7] : 0.f;
#pragma unroll
  for (int d = 4; d > 0; d /= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
  return t;
}

// The whole tile once more from memory where a row of it is not in range, which all blocks of the cluster see alike: such
// rows at their own scale.  A thread has a column.
template <typename TX, typename TH, bool RES>
__device__ __noinline__ void redo_tile(const NormArgs &a, const float (&squares)[32][8]) {
  __shared__ float rstd[32];
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();  // every block's sum is stored
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = int(cluster.num_blocks()), j = int(threadIdx.x);
  const TH *const s = static_cast<const TH *>(RES ? a.sum : a.x);
  const int64_t ld = RES ? a.sum_ld : a.x_ld, row0 = int64_t(blockIdx.y) * 32, c = int64_t(blockIdx.x) * 256 + j;
  const float t = row_squares(squares, blocks);
  for (int i = 0; i < 4; ++i) {
    float sum = __shfl_sync(0xFFFFFFFFu, t, 8 * i), factor = 1.f;
    if (!in_range(a, sum)) {
      factor = factor_of(sum);
      sum = 0.f;
      for (int k = lane; k < int(a.cols); k += 32) {
        const float x = gtp::load1(s + (row0 + 4 * warp + i) * ld + k) * factor;
        sum = fmaf(x, x, sum);
      }
      sum = warp_sum(sum);
    }
    if (lane == 0) rstd[4 * warp + i] = factor == 1.f ? rstd_of(a, sum) : rstd_of(a, sum, factor);
  }
  __syncthreads();
  if (a.rstd && cluster.block_rank() == 0 && j < 32) a.rstd[row0 + j] = rstd[j];
  const bool live = c < a.cols;
  const float w = live ? gtp::load1_of(a.weight, a.weight_f32, c) : 0.f;
  const auto y_of = [&](int i) { return live ? gtp::load1(s + (row0 + i) * ld + c) * rstd[i] * w : 0.f; };
  uint32_t bits = 0;
  for (int i = 0; i < 32; ++i) {
    const float y = y_of(i);
    const uint32_t b = __float_as_uint(y) & 0x7FFFFFFFu;
    bits = max(bits, b);
    const int64_t row = row0 + i;
    if (a.y && live) {
      if (a.y_f32) static_cast<float *>(a.y)[row * a.y_ld + c] = y;
      else static_cast<__nv_bfloat16 *>(a.y)[row * a.y_ld + c] = __float2bfloat16_rn(y);
    }
    if (a.row_codes) {
      float inv;
      const uint32_t byte = block_scale(__reduce_max_sync(0xFFFFFFFFu, b), inv);
      if (live) a.row_codes[row * a.cols + c] = uint8_t(gtp::mx::encode4(y * inv, 0.f, 0.f, 0.f));
      if (live && lane == 0) a.row_scales[scale_at(row, c >> 5, a.cols >> 5, a.row_words)] = uint8_t(byte);
    }
  }
  if (!live) return;
  float inv;
  a.col_scales[scale_at(c, blockIdx.y, a.rows >> 5, a.col_words)] = uint8_t(block_scale(bits, inv));
  for (int i = 0; i < 32; i += 4)
    reinterpret_cast<uint32_t *>(a.col_codes + c * a.rows + row0)[i >> 2] =
        gtp::mx::encode4(y_of(i) * inv, y_of(i + 1) * inv, y_of(i + 2) * inv, y_of(i + 3) * inv);
}

// A block holds 32 rows of 256 columns: its eight warps four rows each, a lane eight columns of every row.  The blocks of
// a cluster share the rows and trade their sums of squares through shared memory.  A column's 32 rows are one block of
// the columnwise view: its amax joins the warps' through shared memory, a lane's four rows are one word of the column's
// 32 bytes.  STATS false: r is read, only the columnwise view is written (rows too wide for a cluster; the sum, r and
// what goes by rows are norm_kernel's).
//
// Both views of [8192, 2048] bf16 with a bf16 residual: 35.5 us, 3.8 TB/s of x, the residual, the sum and the views (36.1
// with the sum written before the cluster's exchange).  Bound by latency: load, exchange and two rounds through shared
// memory follow one another in a block, and four blocks of 64 registers a thread are an SM's (three 38.1 us, five 48.1).
constexpr int kTileThreads = 256, kTileRows = 32, kMostCluster = 8;

// A barrier of the cluster in two halves and without an ordering of memory, by warps whose lanes may have parted: after the
// wait every block of the cluster has come to its arrive, so that its shared memory may be written to.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <typename TX, typename TS, bool RES, bool STATS>
__global__ void __launch_bounds__(kTileThreads, 4) norm_tile_kernel(const __grid_constant__ NormArgs a) {
  constexpr int CW = 256;  // columns
  using TH = typename std::conditional<RES, TS, TX>::type;
  __shared__ __align__(16) uint32_t plane[8][CW];  // columns' amax of each warp, then their codes of each warp's rows
  __shared__ __align__(16) float inv[CW];
  __shared__ float squares[kTileRows][kMostCluster];
  __shared__ int odd;  // a row is not in range
  if (STATS) cluster_arrive_relaxed();
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 = int64_t(blockIdx.y) * kTileRows + 4 * warp, c0 = int64_t(blockIdx.x) * CW;
  Eight<TX> x[4];
  Eight<TH> h[4];
  const int64_t c = c0 + 8 * lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i].clear();
    h[i].clear();
    if (c < a.cols) {
      x[i].load(static_cast<const TX *>(a.x) + (row0 + i) * a.x_ld + c);
      if (RES) h[i].load(static_cast<const TH *>(a.residual) + (row0 + i) * a.residual_ld + c);
    }
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
    x[i].get(f);
    if (RES) {
      float res[8];
      h[i].get(res);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += res[k];
    }
    h[i].set(f);
    if (STATS) {
      h[i].get(f);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[i] = fmaf(f[k], f[k], s[i]);
    }
  }
  const bool live = c < a.cols;
  float r[4], w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = 0.f;
  if (STATS) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), blocks = int(cluster.num_blocks());
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = warp_sum(s[i]);
    cluster_wait();  // the other blocks run, and have their shared memory
    if (lane < blocks) {
      float *const there = cluster.map_shared_rank(&squares[4 * warp][rank], lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) there[i * kMostCluster] = s[i];
    }
    if (threadIdx.x == 0) odd = 0;
    auto token = cluster.barrier_arrive();  // the sum and the weight while the other blocks come
    if (RES && live) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i].store(static_cast<TH *>(a.sum) + (row0 + i) * a.sum_ld + c);
    }
    if (live) gtp::load8_of(a.weight, a.weight_f32, c, w);
    cluster.barrier_wait(std::move(token));
    const float t = row_squares(squares, blocks);
    if (!in_range(a, t)) odd = 1;
    const float rt = rstd_of(a, t);
    if (a.rstd && rank == 0 && (lane & 7) == 0) a.rstd[row0 + (lane >> 3)] = rt;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __shfl_sync(0xFFFFFFFFu, rt, 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = a.rstd[row0 + i];
    if (live) gtp::load8_of(a.weight, a.weight_f32, c, w);
  }
  uint32_t amax[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) amax[k] = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[8];
    h[i].get(y);
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[k] = y[k] * r[i] * w[k];
      const uint32_t b = __float_as_uint(y[k]) & 0x7FFFFFFFu;
      amax[k] = max(amax[k], b);
      bits = max(bits, b);
    }
    if (STATS && a.y && live) store_y(a, row0 + i, c, y);
    if (STATS && a.row_codes) store_row_view(a, row0 + i, c, live, y, bits);
  }
  uint4 *const p = reinterpret_cast<uint4 *>(&plane[warp][8 * lane]);
  p[0] = make_uint4(amax[0], amax[1], amax[2], amax[3]);
  p[1] = make_uint4(amax[4], amax[5], amax[6], amax[7]);
  __syncthreads();
  const int j = threadIdx.x;
  uint32_t bits = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) bits = max(bits, plane[q][j]);
  const uint32_t byte = block_scale(bits, inv[j]);
  if (c0 + j < a.cols) a.col_scales[scale_at(c0 + j, blockIdx.y, a.rows >> 5, a.col_words)] = uint8_t(byte);
  __syncthreads();
  float f[8], y[4][8];
  if (live) gtp::load8_of(a.weight, a.weight_f32, c, w);  // again, as y: not kept over the barriers
  gtp::load8_of(inv, 1, 8 * lane, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // the same y again, from registers
    h[i].get(y[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[i][k] = y[i][k] * r[i] * w[k] * f[k];
  }
  uint32_t code[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) code[k] = gtp::mx::encode4(y[0][k], y[1][k], y[2][k], y[3][k]);
  p[0] = make_uint4(code[0], code[1], code[2], code[3]);
  p[1] = make_uint4(code[4], code[5], code[6], code[7]);
  __syncthreads();
  if (c0 + j < a.cols) {
    uint8_t *const dst = a.col_codes + (c0 + j) * a.rows + int64_t(blockIdx.y) * kTileRows;
    const uint32_t bytes[8] = {plane[0][j], plane[1][j], plane[2][j], plane[3][j],
                               plane[4][j], plane[5][j], plane[6][j], plane[7][j]};
    if (a.codes_on_32) {
      gtp::store_32b(dst, bytes);
    } else {
      reinterpret_cast<uint4 *>(dst)[0] = make_uint4(bytes[0], bytes[1], bytes[2], bytes[3]);
      reinterpret_cast<uint4 *>(dst)[1] = make_uint4(bytes[4], bytes[5], bytes[6], bytes[7]);
    }
  }
  if (STATS && odd) redo_tile<TX, TH, RES>(a, squares);
}

// --------------------------------------------------------------------------- MXFP8 values

// A thread has eight columns, N rows at a time in flight.
template <typename TO>
__global__ void __launch_bounds__(256)
    mxfp8_dequantize_kernel(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, int64_t words, TO *out,
                            int vec) {
  constexpr int N = 4;
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int64_t c = 8 * (int64_t(blockIdx.x) * blockDim.x + threadIdx.x), step = int64_t(gridDim.y) * blockDim.y;
  if (c >= cols) return;
  for (int64_t r0 = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; r0 < rows; r0 += N * step) {
    uint2 q[N];
    uint32_t byte[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step;
      if (row < rows) {
        q[i] = *reinterpret_cast<const uint2 *>(codes + row * cols + c);
        byte[i] = scales[scale_at(row, c >> 5, cols >> 5, words)];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step;
      if (row >= rows) continue;
      // 2^(byte - 127); byte 0 is a subnormal of fp32, 255 NaN
      const float s = byte[i] == 0 ? __uint_as_float(0x00400000u) : byte[i] == 255 ? __uint_as_float(0x7FC00000u)
                                                                                  : __uint_as_float(byte[i] << 23);
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = k < 2 ? q[i].x : q[i].y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * (k & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * k] = f.x * s;
        x[2 * k + 1] = f.y * s;
      }
      TO *const to = out + row * cols + c;
      if (vec) {
        Eight<TO> e;
        e.set(x);
        e.store(to);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) gtp::store1(to + k, x[k]);
      }
    }
  }
}

// --------------------------------------------------------------------------- host

// Threads a row, rows a block, groups of eight a thread: one group up to 4096 columns ([8192, 4096] bf16 42.6 us, with four
// a thread 45.0; [8192, 2048] 22.7 and 23.5), else four ([8192, 5120] 55.8, 8192 columns 85.8).
struct RowShape {
  int tx, ty, V;
};

RowShape row_shape(int64_t cols) {
  const int64_t groups = (cols + 7) / 8;
  const int V = groups <= kRowThreads ? 1 : 4;
  const int tx = int((groups + 32 * V - 1) / (32 * V)) * 32;
  return {tx, tx == 32 ? 8 : 1, V};
}

template <typename TX, typename TS, bool RES>
gtp_status launch_rows(const NormArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const RowShape s = row_shape(a.cols);
  const dim3 block(s.tx, s.ty);
  const int64_t blocks = (a.rows + s.ty - 1) / s.ty, most = int64_t(dev.sm_count) * std::max(1, 2048 / (s.tx * s.ty));
  // rows a time: four of bf16 ([8192, 2048] with a residual 22.7 us, one at a time 26.8), one where a row has more bytes (all
  // fp32 36.3 us, two at a time 40.0); few rows: one, spread over the machine
  constexpr int MANY = sizeof(TX) + (RES ? sizeof(TS) : 0) > 4 ? 1 : 4;
  if (MANY > 1 && s.V == 1 && blocks > most)
    return gtp::launch_overlapped(norm_kernel<TX, TS, RES, 1, MANY>, unsigned((blocks + MANY - 1) / MANY), block, 0, st, "rmsnorm", a);
  return gtp::launch_overlapped(s.V == 1 ? norm_kernel<TX, TS, RES, 1, 1> : norm_kernel<TX, TS, RES, 4, 1>,
                                unsigned(std::min(blocks, most)), block, 0, st, "rmsnorm", a);
}

template <typename TX, typename TS, bool RES, int T, int K>
gtp_status launch_elements_of(const NormArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const dim3 block(T, T == 32 ? 8 : 1);
  const int64_t blocks = (a.rows + block.y - 1) / block.y;
  return gtp::launch_overlapped(norm_elements_kernel<TX, TS, RES, T, K>,
                                unsigned(std::min<int64_t>(blocks, int64_t(dev.sm_count) * 64)), block, 0, st, "rmsnorm", a);
}

// A row is in registers after one round of loads, eight elements a thread, above 2048 columns sixteen ([8192, 4095] 65 us
// with 256 threads of sixteen, 73 with 512 of eight; [8192, 8001] 132 with 512 and 194 with 1024): more blocks an SM are
// worth more than more threads a row ([8192, 1000] 26.2 us with 256 threads, 59.4 with 512; rows of 250 by a warp each 6
// us, by 256 threads 25).
template <typename TX, typename TS, bool RES>
gtp_status launch_elements(const NormArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (a.cols <= 32 * 8) return launch_elements_of<TX, TS, RES, 32, 8>(a, dev, st);
  if (a.cols <= 256 * 8) return launch_elements_of<TX, TS, RES, 256, 8>(a, dev, st);
  if (a.cols <= 256 * 16) return launch_elements_of<TX, TS, RES, 256, 16>(a, dev, st);
  if (a.cols <= 512 * 16) return launch_elements_of<TX, TS, RES, 512, 16>(a, dev, st);
  return launch_elements_of<TX, TS, RES, 1024, 16>(a, dev, st);
}

template <typename TX, typename TS, bool RES, bool STATS>
gtp_status launch_tiles_of(const NormArgs &a, cudaStream_t st) {
  const int64_t wide = (a.cols + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(wide), unsigned(a.rows / kTileRows));
  cfg.blockDim = dim3(kTileThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (!std::getenv("GTP_NO_LAUNCH_OVERLAP")) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (STATS) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(wide);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(n);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_tile_kernel<TX, TS, RES, STATS>, a);
  if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "rmsnorm: %s", cudaGetErrorString(e));
  return gtp::check_launch("rmsnorm");
}

template <typename TX, typename TS, bool RES>
gtp_status launch_tiles(NormArgs a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  // one launch where a cluster holds a row: [8192, 2048] with a bf16 residual 35.3 us and by two launches 35.4, with an fp32 one
  // 44.3 and 47.4, without 29.1 and 32.3; [256, 2048] 5.2 and 6.4.  Two above: [8192, 4096] 67.4, where a cluster of eight
  // blocks of 512 columns took 76 to 79
  if (a.cols <= 256 * kMostCluster) return launch_tiles_of<TX, TS, RES, true>(a, st);
  uint8_t *const codes = a.col_codes;
  a.col_codes = nullptr;
  if (gtp_status s = launch_rows<TX, TS, RES>(a, dev, st)) return s;
  a.col_codes = codes;
  if (RES) a.x = a.sum, a.x_ld = a.sum_ld;
  return launch_tiles_of<TS, TS, false, false>(a, st);
}

template <typename TX, typename TS, bool RES>
gtp_status launch(const NormArgs &a, bool vec, const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (a.col_codes) return launch_tiles<TX, TS, RES>(a, dev, st);
  return vec ? launch_rows<TX, TS, RES>(a, dev, st) : launch_elements<TX, TS, RES>(a, dev, st);
}

}  // namespace

extern "C" gtp_status gtp_rmsnorm(const gtp_rmsnorm_desc *d, gtp_stream stream) {
  gtp::clear_error();
  if (!d) return gtp::fail(GTP_E_ARG, "null descriptor");
  const bool res = d->residual != nullptr, row_view = d->row_codes || d->row_scales, col_view = d->col_codes || d->col_scales;
  if (d->reserved) return gtp::fail(GTP_E_ARG, "reserved must be 0");
  if ((d->tiled_scales != 0 && d->tiled_scales != 1) || !(d->eps >= 0.f) || std::isinf(d->eps))
    return gtp::fail(GTP_E_ARG, "tiled_scales must be 0 or 1, eps finite and not negative");
  if (!float_type(d->x_dtype) || !float_type(d->weight_dtype) || (res && !float_type(d->residual_dtype)) ||
      (d->y && !float_type(d->y_dtype)))
    return gtp::fail(GTP_E_DTYPE, "dtypes must be F32 or BF16");
  if (d->rows < 0 || d->cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (d->rows > kMaxRows || d->cols > kMaxCols) return gtp::fail(GTP_E_SHAPE, "rows above 2^30 or cols above 16384");
  if ((row_view && d->cols % 32) || (col_view && (d->rows % 32 || d->cols % 32)))
    return gtp::fail(GTP_E_SHAPE, "a view needs whole blocks of 32: cols, and rows for the columnwise view");
  if (col_view && d->rows / 32 > 65535) return gtp::fail(GTP_E_SHAPE, "rows / 32 above 65535 with a columnwise view");
  if (d->rows == 0 || d->cols == 0) return GTP_OK;
  if (res != (d->sum != nullptr)) return gtp::fail(GTP_E_ARG, "residual and sum are given together");
  if (!d->y && !row_view && !col_view && !res && !d->rstd) return gtp::fail(GTP_E_ARG, "no output");
  if ((row_view && !(d->row_codes && d->row_scales)) || (col_view && !(d->col_codes && d->col_scales)))
    return gtp::fail(GTP_E_ARG, "a view's codes and scales are given together");
  if (col_view && !d->rstd) return gtp::fail(GTP_E_ARG, "the columnwise view needs rstd");
  const int64_t R = d->rows, C = d->cols;
  const Matrix x = {"x", d->x, d->x_ld, d->x_dtype}, r = {"residual", d->residual, d->residual_ld, d->residual_dtype},
               s = {"sum", d->sum, d->sum_ld, d->residual_dtype}, y = {"y", d->y, d->y_ld, d->y_dtype},
               w = {"weight", d->weight, C, d->weight_dtype};
  if (gtp_status e = check_matrix(x, R, C)) return e;
  if (gtp_status e = check_matrix(w, 1, C)) return e;
  if (res)
    for (const Matrix *m : {&r, &s})
      if (gtp_status e = check_matrix(*m, R, C)) return e;
  if (d->y)
    if (gtp_status e = check_matrix(y, R, C)) return e;
  if (d->rstd && !aligned(d->rstd, 4)) return gtp::fail(GTP_E_ALIGN, "rstd must be 4-byte aligned");
  bool vec = C % 8 == 0 && vector_rows(x, R) && aligned(w.p, 16);
  if (res) vec = vec && vector_rows(r, R) && vector_rows(s, R);
  if (d->y) vec = vec && vector_rows(y, R);
  if ((row_view || col_view) && (!vec || !aligned(d->row_codes, 16) || !aligned(d->col_codes, 16)))
    return gtp::fail(GTP_E_ALIGN, "with a view the rows of every matrix start on eight elements, the weight and the codes on 16 bytes");
  // no output shares a byte with an input or another output, but for the sum in place of x or of the residual, and y in
  // place of x
  gtp::Runs out[7];
  const Matrix *place[7];
  int n = 0;
  const auto add = [&](const gtp::Runs &runs, const Matrix *m) { out[n] = runs, place[n++] = m; };
  const int64_t row_bytes = gtp_sf_tiled_bytes(R, C / 32), col_bytes = gtp_sf_tiled_bytes(C, R / 32);
  if (res) add(runs_of(s, R, C), &s);
  if (d->y) add(runs_of(y, R, C), &y);
  if (d->rstd) add(runs_of(d->rstd, 4 * R), nullptr);
  if (row_view) {
    add(runs_of(d->row_codes, R * C), nullptr);
    add(runs_of(d->row_scales, d->tiled_scales ? row_bytes : R * (C / 32)), nullptr);
  }
  if (col_view) {
    add(runs_of(d->col_codes, R * C), nullptr);
    add(runs_of(d->col_scales, d->tiled_scales ? col_bytes : C * (R / 32)), nullptr);
  }
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < i; ++j)
      if (gtp::overlap(out[i], out[j])) return gtp::fail(GTP_E_ARG, "two outputs overlap");
    if (gtp::overlap(out[i], runs_of(w, 1, C))) return gtp::fail(GTP_E_ARG, "an output overlaps the weight");
    if (!(place[i] && same_place(*place[i], x, R)) && gtp::overlap(out[i], runs_of(x, R, C)))
      return gtp::fail(GTP_E_ARG, "an output overlaps x and is not it");
    if (res && !(place[i] == &s && same_place(s, r, R)) && gtp::overlap(out[i], runs_of(r, R, C)))
      return gtp::fail(GTP_E_ARG, "an output overlaps the residual and is not it");
  }
  if (col_view && !res && d->y && same_place(y, x, R))
    return gtp::fail(GTP_E_ARG, "y in place of x with a columnwise view");
  gtp::DeviceInfo dev;
  if (gtp_status e = gtp::require_sm103(&dev)) return e;
  NormArgs a = {};
  a.x = d->x, a.residual = d->residual, a.weight = d->weight, a.sum = d->sum, a.y = d->y, a.rstd = d->rstd;
  a.row_codes = d->row_codes, a.row_scales = d->row_scales, a.col_codes = d->col_codes, a.col_scales = d->col_scales;
  a.rows = R, a.cols = C;
  a.x_ld = R > 1 ? d->x_ld : C, a.residual_ld = R > 1 ? d->residual_ld : C;
  a.sum_ld = R > 1 ? d->sum_ld : C, a.y_ld = R > 1 ? d->y_ld : C;
  a.row_words = d->tiled_scales ? (C / 32 + 3) / 4 : 0;
  a.col_words = d->tiled_scales ? (R / 32 + 3) / 4 : 0;
  a.inv_cols = 1.f / float(C), a.codes_on_32 = aligned(d->col_codes, 32);
  // a mean that the squares' last bits, 2^-149 each, do not reach in any case is left alone
  a.eps = d->eps, a.least = d->eps >= 0x1p-80f ? 0.f : 0x1p-100f;
  a.weight_f32 = d->weight_dtype == GTP_F32, a.y_f32 = d->y_dtype == GTP_F32;
  cudaStream_t st = gtp::as_stream(stream);
  using B = __nv_bfloat16;
  if (!res) return d->x_dtype == GTP_F32 ? launch<float, float, false>(a, vec, dev, st) : launch<B, B, false>(a, vec, dev, st);
  if (d->residual_dtype == GTP_F32)
    return d->x_dtype == GTP_F32 ? launch<float, float, true>(a, vec, dev, st) : launch<B, float, true>(a, vec, dev, st);
  return d->x_dtype == GTP_F32 ? launch<float, B, true>(a, vec, dev, st) : launch<B, B, true>(a, vec, dev, st);
}

extern "C" gtp_status gtp_mxfp8_dequantize(const uint8_t *e4m3, const uint8_t *e8m0, int32_t tiled_scales, int64_t rows,
                                           int64_t cols, void *out, gtp_dtype out_dt, gtp_stream stream) {
  gtp::clear_error();
  if (!float_type(out_dt)) return gtp::fail(GTP_E_DTYPE, "out must be F32 or BF16");
  if (tiled_scales != 0 && tiled_scales != 1) return gtp::fail(GTP_E_ARG, "tiled_scales must be 0 or 1");
  if (rows < 0 || cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (rows > kMaxRows || cols > kMaxRows || rows > (int64_t(1) << 40) / std::max<int64_t>(cols, 1))
    return gtp::fail(GTP_E_SHAPE, "a dimension above 2^30 or more than 2^40 elements");
  if (cols % 32) return gtp::fail(GTP_E_SHAPE, "cols must be a multiple of 32");
  if (rows == 0 || cols == 0) return GTP_OK;
  if (!e4m3 || !e8m0 || !out) return gtp::fail(GTP_E_ARG, "null pointer");
  if (!aligned(e4m3, 16) || !aligned(out, size_of(out_dt)))
    return gtp::fail(GTP_E_ALIGN, "codes must be 16-byte aligned, out to its elements");
  const gtp::ByteRange o = gtp::byte_range(out, rows * cols * size_of(out_dt));
  if (gtp::overlap(o, gtp::byte_range(e4m3, rows * cols)) ||
      gtp::overlap(o, gtp::byte_range(e8m0, tiled_scales ? gtp_sf_tiled_bytes(rows, cols / 32) : rows * (cols / 32))))
    return gtp::fail(GTP_E_ARG, "out overlaps the view");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  const int64_t words = tiled_scales ? (cols / 32 + 3) / 4 : 0;
  int tx = 4;
  while (tx < 256 && 8 * tx < cols) tx *= 2;
  const dim3 block(tx, 256 / tx);
  const int64_t gx = (cols + 8 * tx - 1) / (8 * tx);
  const dim3 grid(unsigned(gx), unsigned(std::min<int64_t>((rows + 4 * block.y - 1) / (4 * block.y), 65535)));
  cudaStream_t st = gtp::as_stream(stream);
  const int vec = aligned(out, 8 * size_of(out_dt));
  if (out_dt == GTP_F32)
    return gtp::launch_overlapped(mxfp8_dequantize_kernel<float>, grid, block, 0, st, "mxfp8_dequantize", e4m3, e8m0, rows, cols,
                                  words, static_cast<float *>(out), vec);
  return gtp::launch_overlapped(mxfp8_dequantize_kernel<__nv_bfloat16>, grid, block, 0, st, "mxfp8_dequantize", e4m3, e8m0, rows,
                                cols, words, static_cast<__nv_bfloat16 *>(out), vec);
}
