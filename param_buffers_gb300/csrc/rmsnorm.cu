// Root-mean-square norm with the residual's addition, its output in bf16 or fp32 and / or as the MXFP8 views that a
// linear's products read, and its gradient, the weight's accumulated into the flat gradient buffer.
//
// Pages: "Megatron-LM architecture and source guide" (arganzheng.life), §1 (the transformer layer: a norm before the
// attention block and before the MLP, each on the residual stream); "Generalized Tensor Parallelism (GTP)"
// (Megatron-Core developer guide), §1.3 (MXFP8 rowwise and columnwise views).
//
//   s = x + residual (rounded to the stream's type; s = x without one)     r = 1 / sqrt(mean s^2 + eps) per row
//   y = (s r) w                                                             views: MXFP8 of the fp32 y, one rounding
//   n = s r, g = dy w:   dx = r (g - n mean(g n)) + dsum                    dw += sum over rows of dy n
// Sums in fp32.  Everything is bound by the bytes: one pass over them, a row's elements staying in registers between
// the sum of squares and the outputs.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "byte_range.h"
#include "device.h"
#include "mx_block.cuh"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

namespace cg = cooperative_groups;

// Eight elements that one thread moves: consecutive ones on 16 bytes (VEC), or every step-th from its own on, so that a
// warp's accesses stay side by side whatever a row's alignment; n of them exist.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int step, int n, float (&x)[8]) {
  if (VEC) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);  // bf16 -> fp32 is exact
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? __bfloat162float(p[k * step]) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float *p, int step, int n, float (&x)[8]) {
  if (VEC) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k * step] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int step, int n, const float (&x)[8]) {
  if (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k * step] = __float2bfloat16_rn(x[k]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, int step, int n, const float (&x)[8]) {
  if (VEC) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k * step] = x[k];
  }
}
__device__ __forceinline__ float rounded(float v, float) { return v; }
__device__ __forceinline__ float rounded(float v, __nv_bfloat16) { return __bfloat162float(__float2bfloat16_rn(v)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

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
  float eps;
  int weight_f32, y_f32;
};

template <bool VEC>
__device__ __forceinline__ void load_weight(const void *w, int f32, int64_t c, int step, int n, float (&x)[8]) {
  if (f32) load8<VEC>(static_cast<const float *>(w) + c, step, n, x);
  else load8<VEC>(static_cast<const __nv_bfloat16 *>(w) + c, step, n, x);
}

template <bool VEC>
__device__ __forceinline__ void store_y(const NormArgs &a, int64_t row, int64_t c, int step, int n, const float (&y)[8]) {
  if (a.y_f32) store8<VEC>(static_cast<float *>(a.y) + row * a.y_ld + c, step, n, y);
  else store8<VEC>(static_cast<__nv_bfloat16 *>(a.y) + row * a.y_ld + c, step, n, y);
}

// The rowwise view of eight consecutive elements of a row: four lanes hold a block.  All 32 lanes take part; live: this
// one's elements exist (whole blocks do or do not).
__device__ __forceinline__ void store_row_view(const NormArgs &a, int64_t row, int64_t c, bool live, const float (&y)[8]) {
  uint32_t bits = 0;  // the largest |y| pattern: the amax, and above every finite one's where there is NaN or Inf
#pragma unroll
  for (int k = 0; k < 8; ++k) bits = max(bits, __float_as_uint(y[k]) & 0x7FFFFFFFu);
  bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
  bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 2));
  if (!live) return;
  uint32_t byte = gtp::mx::kNanScale;
  uint2 codes = make_uint2(gtp::mx::kNanCodes, gtp::mx::kNanCodes);
  if (bits < 0x7F800000u) {
    byte = gtp::mx::scale_byte(__uint_as_float(bits));
    const float inv = gtp::mx::inv_scale(byte);
    codes.x = gtp::mx::encode4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    codes.y = gtp::mx::encode4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
  }
  *reinterpret_cast<uint2 *>(a.row_codes + row * a.cols + c) = codes;
  if ((c & 31) == 0) a.row_scales[scale_at(row, c >> 5, a.cols >> 5, a.row_words)] = uint8_t(byte);
}

// --------------------------------------------------------------------------- forward, row by row

// blockDim.x threads a row (whole warps), V groups of eight elements a thread, blockDim.y rows a block.  Without VEC
// group v holds elements (8 v + k) blockDim.x + threadIdx.x.
template <typename TX, typename TS, bool RES, bool VEC, int V>
__global__ void __launch_bounds__(kRowThreads) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int tx = blockDim.x, lane = threadIdx.x & 31, warps = tx >> 5;
  int flip = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < a.rows; r0 += int64_t(gridDim.x) * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < a.rows;
    float h[V][8];
    float squares = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = VEC ? 8 * (int64_t(v) * tx + threadIdx.x) : int64_t(v) * 8 * tx + threadIdx.x;
      const int n = c >= a.cols || !live ? 0 : VEC ? 8 : int(min(int64_t(8), (a.cols - c + tx - 1) / tx));
      if (n > 0) {
        load8<VEC>(static_cast<const TX *>(a.x) + row * a.x_ld + c, tx, n, h[v]);
        if (RES) {
          float res[8];
          load8<VEC>(static_cast<const TS *>(a.residual) + row * a.residual_ld + c, tx, n, res);
#pragma unroll
          for (int k = 0; k < 8; ++k) h[v][k] = rounded(h[v][k] + res[k], TS());
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) h[v][k] = 0.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = VEC ? 8 * (int64_t(v) * tx + threadIdx.x) : int64_t(v) * 8 * tx + threadIdx.x;
      const int n = c >= a.cols || !live ? 0 : VEC ? 8 : int(min(int64_t(8), (a.cols - c + tx - 1) / tx));
      if (RES && n > 0) store8<VEC>(static_cast<TS *>(a.sum) + row * a.sum_ld + c, tx, n, h[v]);
#pragma unroll
      for (int k = 0; k < 8; ++k) squares = fmaf(h[v][k], h[v][k], squares);
    }
    squares = warp_sum(squares);
    if (warps > 1) {  // one row a block then; the two arrays let one barrier a row do
      if (lane == 0) part[flip][threadIdx.x >> 5] = squares;
      __syncthreads();
      squares = warp_sum(lane < warps ? part[flip][lane] : 0.f);
    }
    const float r = 1.f / sqrtf(squares / float(a.cols) + a.eps);
    if (a.rstd && live && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = VEC ? 8 * (int64_t(v) * tx + threadIdx.x) : int64_t(v) * 8 * tx + threadIdx.x;
      const int n = c >= a.cols || !live ? 0 : VEC ? 8 : int(min(int64_t(8), (a.cols - c + tx - 1) / tx));
      float y[8];
      if (n > 0) load_weight<VEC>(a.weight, a.weight_f32, c, tx, n, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = n > 0 ? h[v][k] * r * y[k] : 0.f;
      if (a.y && n > 0) store_y<VEC>(a, row, c, tx, n, y);
      if (VEC && a.row_codes) store_row_view(a, row, c, n > 0, y);
    }
  }
}

// --------------------------------------------------------------------------- forward with the columnwise view

// A block holds 32 rows of 256 VPL columns: its eight warps four rows each, a lane VPL vectors of eight columns of every
// row.  The blocks of a cluster share the rows and trade their sums of squares through shared memory.  A column's 32
// rows are one block of the columnwise view: its amax joins the warps' through shared memory, a lane's four rows are
// one word of the column's 32 bytes.  STATS false: r is read, only the columnwise view is written (rows too wide for a
// cluster; the sum, r and what goes by rows are norm_kernel's).
constexpr int kTileThreads = 256, kTileRows = 32, kMostCluster = 8;

template <typename TX, typename TS, bool RES, int VPL, bool STATS>
__global__ void __launch_bounds__(kTileThreads) norm_tile_kernel(const __grid_constant__ NormArgs a) {
  constexpr int CW = 256 * VPL;
  __shared__ __align__(16) uint32_t plane[8][CW];  // columns' amax of each warp, then their codes of each warp's rows
  __shared__ __align__(16) float inv[CW];
  __shared__ uint8_t bad[CW];
  __shared__ float squares[kMostCluster][kTileRows];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 = int64_t(blockIdx.y) * kTileRows + 4 * warp, c0 = int64_t(blockIdx.x) * CW;
  float h[4][VPL][8], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int64_t c = c0 + 8 * (32 * v + lane);
      if (c < a.cols) {
        load8<true>(static_cast<const TX *>(a.x) + (row0 + i) * a.x_ld + c, 1, 8, h[i][v]);
        if (RES) {
          float res[8];
          load8<true>(static_cast<const TS *>(a.residual) + (row0 + i) * a.residual_ld + c, 1, 8, res);
#pragma unroll
          for (int k = 0; k < 8; ++k) h[i][v][k] = rounded(h[i][v][k] + res[k], TS());
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][v][k] = 0.f;
      }
    }
  }
  if (STATS) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), blocks = int(cluster.num_blocks());
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(h[i][v][k], h[i][v][k], s);
      s = warp_sum(s);
      if (lane < blocks) *cluster.map_shared_rank(&squares[rank][4 * warp + i], lane) = s;
    }
    cluster.sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s = 0.f;
      for (int b = 0; b < blocks; ++b) s += squares[b][4 * warp + i];  // the same order in every block
      r[i] = 1.f / sqrtf(s / float(a.cols) + a.eps);
      if (a.rstd && rank == 0 && lane == 0) a.rstd[row0 + i] = r[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = a.rstd[row0 + i];
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int64_t c = c0 + 8 * (32 * v + lane);
    const bool live = c < a.cols;
    float w[8];
    uint32_t amax[8];
    if (live) load_weight<true>(a.weight, a.weight_f32, c, 1, 8, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) amax[k] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (STATS && RES && live) store8<true>(static_cast<TS *>(a.sum) + (row0 + i) * a.sum_ld + c, 1, 8, h[i][v]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][v][k] = live ? h[i][v][k] * r[i] * w[k] : 0.f;  // y from here on
        amax[k] = max(amax[k], __float_as_uint(h[i][v][k]) & 0x7FFFFFFFu);
      }
      if (STATS && a.y && live) store_y<true>(a, row0 + i, c, 1, 8, h[i][v]);
      if (STATS && a.row_codes) store_row_view(a, row0 + i, c, live, h[i][v]);
    }
    uint4 *p = reinterpret_cast<uint4 *>(&plane[warp][8 * (32 * v + lane)]);
    p[0] = make_uint4(amax[0], amax[1], amax[2], amax[3]);
    p[1] = make_uint4(amax[4], amax[5], amax[6], amax[7]);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int j = 256 * v + threadIdx.x;
    uint32_t bits = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) bits = max(bits, plane[w][j]);
    const bool finite = bits < 0x7F800000u;
    const uint32_t byte = finite ? gtp::mx::scale_byte(__uint_as_float(bits)) : gtp::mx::kNanScale;
    inv[j] = finite ? gtp::mx::inv_scale(byte) : 0.f;
    bad[j] = finite ? 0 : 1;
    if (c0 + j < a.cols) a.col_scales[scale_at(c0 + j, blockIdx.y, a.rows >> 5, a.col_words)] = uint8_t(byte);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int j = 8 * (32 * v + lane);
    uint32_t code[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = inv[j + k];
      code[k] = bad[j + k] ? gtp::mx::kNanCodes
                           : gtp::mx::encode4(h[0][v][k] * s, h[1][v][k] * s, h[2][v][k] * s, h[3][v][k] * s);
    }
    uint4 *p = reinterpret_cast<uint4 *>(&plane[warp][j]);
    p[0] = make_uint4(code[0], code[1], code[2], code[3]);
    p[1] = make_uint4(code[4], code[5], code[6], code[7]);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int j = 256 * v + threadIdx.x;
    if (c0 + j < a.cols) {
      uint4 *dst = reinterpret_cast<uint4 *>(a.col_codes + (c0 + j) * a.rows + int64_t(blockIdx.y) * kTileRows);
      dst[0] = make_uint4(plane[0][j], plane[1][j], plane[2][j], plane[3][j]);
      dst[1] = make_uint4(plane[4][j], plane[5][j], plane[6][j], plane[7][j]);
    }
  }
}

// --------------------------------------------------------------------------- gradient

struct GradArgs {
  const void *dy, *sum, *weight, *dsum;
  const float *rstd;
  void *dx;
  float *part;  // [gridDim.x * blockDim.y][cols]: the weight's gradient of each place's rows
  int64_t rows, cols, dy_ld, sum_ld, dsum_ld, dx_ld;
  int weight_f32;
};

// A thread keeps its columns over all its rows, so that their weight and their part of the weight's gradient stay in
// registers; N rows at a time share a barrier and have their loads in flight together.
template <typename TD, typename TS, bool VEC, int V>
__global__ void __launch_bounds__(kRowThreads) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  constexpr int N = V == 1 ? 2 : 1;
  __shared__ float part[2][N][32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int tx = blockDim.x, lane = threadIdx.x & 31, warps = tx >> 5;
  constexpr bool KEEP = V < 4;  // the weight in registers
  float w[KEEP ? V : 1][8], dw[V][8];
  int64_t c[V];
  int n[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = VEC ? 8 * (int64_t(v) * tx + threadIdx.x) : int64_t(v) * 8 * tx + threadIdx.x;
    n[v] = c[v] >= a.cols ? 0 : VEC ? 8 : int(min(int64_t(8), (a.cols - c[v] + tx - 1) / tx));
#pragma unroll
    for (int k = 0; k < 8; ++k) w[KEEP ? v : 0][k] = dw[v][k] = 0.f;
    if (KEEP && n[v] > 0) load_weight<VEC>(a.weight, a.weight_f32, c[v], tx, n[v], w[KEEP ? v : 0]);
  }
  int flip = 0;
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < a.rows; r0 += N * step, flip ^= 1) {
    float g[N][V][8], h[N][V][8], r[N], dot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step + threadIdx.y;
      const bool live = row < a.rows;
      r[i] = live ? a.rstd[row] : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (n[v] > 0 && live) {
          load8<VEC>(static_cast<const TD *>(a.dy) + row * a.dy_ld + c[v], tx, n[v], g[i][v]);
          load8<VEC>(static_cast<const TS *>(a.sum) + row * a.sum_ld + c[v], tx, n[v], h[i][v]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) g[i][v][k] = h[i][v][k] = 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dot[i] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!KEEP && n[v] > 0) load_weight<VEC>(a.weight, a.weight_f32, c[v], tx, n[v], w[0]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[i][v][k] *= r[i];  // n
          dw[v][k] = fmaf(g[i][v][k], h[i][v][k], dw[v][k]);
          g[i][v][k] *= w[KEEP ? v : 0][k];
          dot[i] = fmaf(g[i][v][k], h[i][v][k], dot[i]);
        }
      }
      dot[i] = warp_sum(dot[i]);
    }
    if (warps > 1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane == 0) part[flip][i][threadIdx.x >> 5] = dot[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) dot[i] = warp_sum(lane < warps ? part[flip][i][lane] : 0.f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step + threadIdx.y;
      if (row >= a.rows) continue;
      const float mean = dot[i] / float(a.cols);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (n[v] == 0) continue;
        float d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = 0.f;
        if (a.dsum) load8<VEC>(static_cast<const TS *>(a.dsum) + row * a.dsum_ld + c[v], tx, n[v], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float t = fmaf(-h[i][v][k], mean, g[i][v][k]);
          d[k] = fmaf(r[i], t, d[k]);
        }
        store8<VEC>(static_cast<TS *>(a.dx) + row * a.dx_ld + c[v], tx, n[v], d);
      }
    }
  }
  float *const out = a.part + (int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * a.cols;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (n[v] > 0) store8<false>(out + c[v], VEC ? 1 : tx, n[v], dw[v]);
}

// grad[c] += sum of the parts' column c, in a fixed order: 32 columns a block, each by 32 threads in turn.
template <typename TG>
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float *part, int parts, int64_t cols, TG *grad) {
  __shared__ float sums[32][33];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int p = threadIdx.y; p < parts; p += 32) s += part[int64_t(p) * cols + c];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(sums[threadIdx.x][threadIdx.y]);  // warp y: column y of the block
  const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < cols) {
    if constexpr (sizeof(TG) == 4) grad[col] += s;
    else grad[col] = __float2bfloat16_rn(__bfloat162float(grad[col]) + s);
  }
}

// --------------------------------------------------------------------------- MXFP8 values

template <typename TO>
__global__ void __launch_bounds__(256)
    mxfp8_dequantize_kernel(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, int64_t words, TO *out,
                            int vec) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int64_t blocks = cols >> 5, items = rows * (cols >> 3), step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < items; i += step) {
    const int64_t row = i / (cols >> 3), j = i - row * (cols >> 3);
    const uint2 q = *reinterpret_cast<const uint2 *>(codes + 8 * i);
    const uint32_t byte = scales[scale_at(row, j >> 2, blocks, words)];
    // 2^(byte - 127); byte 0 is a subnormal of fp32, 255 NaN
    const float s = byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7FC00000u)
                                                                          : __uint_as_float(byte << 23);
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? q.x : q.y;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * (k & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      x[2 * k] = f.x * s;
      x[2 * k + 1] = f.y * s;
    }
    if (vec) store8<true>(out + 8 * i, 1, 8, x);
    else store8<false>(out + 8 * i, 1, 8, x);
  }
}

// --------------------------------------------------------------------------- host

int64_t size_of(int dt) { return dt == GTP_F32 ? 4 : 2; }
bool float_type(int dt) { return dt == GTP_F32 || dt == GTP_BF16; }
bool aligned(const void *p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(to - 1)) == 0; }

struct Matrix {
  const char *name;
  const void *p;
  int64_t ld;
  int dt;
};

gtp_status check_matrix(const Matrix &m, int64_t rows, int64_t cols) {
  if (!m.p) return gtp::fail(GTP_E_ARG, "null %s", m.name);
  if (!aligned(m.p, size_of(m.dt))) return gtp::fail(GTP_E_ALIGN, "%s must be aligned to its elements", m.name);
  if (rows > 1 && m.ld < cols) return gtp::fail(GTP_E_ARG, "the row stride of %s is below cols", m.name);
  if (rows > 1 && m.ld > (int64_t(1) << 50) / rows)
    return gtp::fail(GTP_E_SHAPE, "%s spans more than 2^50 elements", m.name);
  return GTP_OK;
}

gtp::Runs runs_of(const Matrix &m, int64_t rows, int64_t cols) {
  const int64_t es = size_of(m.dt);
  return {reinterpret_cast<uintptr_t>(m.p), cols * es, {{(rows > 1 ? m.ld : cols) * es, rows}, {0, 1}, {0, 1}}};
}

gtp::Runs runs_of(const void *p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), bytes, {{bytes, 1}, {0, 1}, {0, 1}}}; }

// Whether `out` may be written where `in` is read by the thread that writes it: the same elements.
bool same_place(const Matrix &out, const Matrix &in, int64_t rows) {
  return out.p == in.p && out.dt == in.dt && (rows == 1 || out.ld == in.ld);
}

bool vector_rows(const Matrix &m, int64_t rows) {
  return aligned(m.p, 16) && (rows == 1 || m.ld * size_of(m.dt) % 16 == 0);
}

// Threads a row and groups of eight a thread.
struct RowShape {
  int tx, ty, V;
};

RowShape row_shape(int64_t rows, int64_t cols, int sms) {
  const int64_t groups = (cols + 7) / 8;
  // few rows: one group a thread, the shortest way through a row; many: more loads in flight a thread, fewer barriers
  int V = rows <= 4 * sms ? 1 : groups > 128 ? 4 : groups > 64 ? 2 : 1;
  while (groups > int64_t(V) * kRowThreads) V *= 2;
  const int tx = int((groups + 32 * V - 1) / (32 * V)) * 32;
  return {tx, tx == 32 ? 8 : 1, V};
}

template <typename TX, typename TS, bool RES, bool VEC>
gtp_status launch_rows(const NormArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const RowShape s = row_shape(a.rows, a.cols, dev.sm_count);
  const dim3 block(s.tx, s.ty);
  const int64_t most = int64_t(dev.sm_count) * std::max(1, 2048 / (s.tx * s.ty));
  const unsigned grid = unsigned(std::min<int64_t>((a.rows + s.ty - 1) / s.ty, most));
  const auto kernel = s.V == 1   ? norm_kernel<TX, TS, RES, VEC, 1>
                      : s.V == 2 ? norm_kernel<TX, TS, RES, VEC, VEC ? 2 : 4>
                                 : norm_kernel<TX, TS, RES, VEC, 4>;
  return gtp::launch_overlapped(kernel, grid, block, 0, st, "rmsnorm", a);
}

template <typename TX, typename TS, bool RES, int VPL, bool STATS>
gtp_status launch_tiles_of(const NormArgs &a, cudaStream_t st) {
  const int64_t wide = (a.cols + 256 * VPL - 1) / (256 * VPL);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_tile_kernel<TX, TS, RES, VPL, STATS>, a);
  if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "rmsnorm: %s", cudaGetErrorString(e));
  return gtp::check_launch("rmsnorm");
}

template <typename TX, typename TS, bool RES>
gtp_status launch_tiles(NormArgs a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (a.cols <= 256 * kMostCluster) return launch_tiles_of<TX, TS, RES, 1, true>(a, st);
  if (a.cols <= 512 * kMostCluster) return launch_tiles_of<TX, TS, RES, 2, true>(a, st);
  uint8_t *const codes = a.col_codes;
  a.col_codes = nullptr;
  if (gtp_status s = launch_rows<TX, TS, RES, true>(a, dev, st)) return s;
  a.col_codes = codes;
  if (RES) a.x = a.sum, a.x_ld = a.sum_ld;
  return launch_tiles_of<TS, TS, false, 1, false>(a, st);
}

template <typename TX, typename TS, bool RES>
gtp_status launch(const NormArgs &a, bool vec, const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (a.col_codes) return launch_tiles<TX, TS, RES>(a, dev, st);
  return vec ? launch_rows<TX, TS, RES, true>(a, dev, st) : launch_rows<TX, TS, RES, false>(a, dev, st);
}

struct GradShape {
  RowShape row;
  int grid;
};

// One rule for the workspace's size and the launch: two blocks of 1024 threads an SM.
GradShape grad_shape(int64_t rows, int64_t cols, int sms) {
  const int64_t groups = (cols + 7) / 8;
  int V = 1;
  while (groups > int64_t(V) * kRowThreads) V *= 2;
  const int tx = int((groups + 32 * V - 1) / (32 * V)) * 32;
  const int ty = tx == 32 ? 8 : 1;
  const int64_t most = int64_t(sms) * std::max(1, (V == 1 ? 1024 : 1024) / (tx * ty));
  return {{tx, ty, V}, int(std::min<int64_t>((rows + ty - 1) / ty, most))};
}

constexpr int kMostSms = 160;  // the workspace's size is asked for without a device: at least an sm_103 GPU's SMs

template <typename TD, typename TS, bool VEC>
gtp_status launch_grad_of(const GradArgs &a, const GradShape &s, cudaStream_t st) {
  const auto kernel = s.row.V == 1   ? norm_grad_kernel<TD, TS, VEC, 1>
                      : s.row.V == 2 ? norm_grad_kernel<TD, TS, VEC, VEC ? 2 : 4>
                                     : norm_grad_kernel<TD, TS, VEC, 4>;
  return gtp::launch_overlapped(kernel, unsigned(s.grid), dim3(s.row.tx, s.row.ty), 0, st, "rmsnorm_grad", a);
}

template <typename TD, typename TS>
gtp_status launch_grad(const GradArgs &a, bool vec, const GradShape &s, cudaStream_t st) {
  return vec ? launch_grad_of<TD, TS, true>(a, s, st) : launch_grad_of<TD, TS, false>(a, s, st);
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
    return gtp::fail(GTP_E_ALIGN, "with a view the rows of every matrix, the weight and the codes start on 16 bytes");
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
  a.eps = d->eps, a.weight_f32 = d->weight_dtype == GTP_F32, a.y_f32 = d->y_dtype == GTP_F32;
  cudaStream_t st = gtp::as_stream(stream);
  using B = __nv_bfloat16;
  if (!res) return d->x_dtype == GTP_F32 ? launch<float, float, false>(a, vec, dev, st) : launch<B, B, false>(a, vec, dev, st);
  if (d->residual_dtype == GTP_F32)
    return d->x_dtype == GTP_F32 ? launch<float, float, true>(a, vec, dev, st) : launch<B, float, true>(a, vec, dev, st);
  return d->x_dtype == GTP_F32 ? launch<float, B, true>(a, vec, dev, st) : launch<B, B, true>(a, vec, dev, st);
}

extern "C" int64_t gtp_rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxCols) return -1;
  if (rows == 0 || cols == 0) return 0;
  const GradShape s = grad_shape(rows, cols, kMostSms);
  return int64_t(s.grid) * s.row.ty * cols * 4;
}

extern "C" gtp_status gtp_rmsnorm_grad(const gtp_rmsnorm_grad_desc *d, void *workspace, int64_t workspace_bytes,
                                       gtp_stream stream) {
  gtp::clear_error();
  if (!d) return gtp::fail(GTP_E_ARG, "null descriptor");
  if (d->reserved) return gtp::fail(GTP_E_ARG, "reserved must be 0");
  if (!float_type(d->dy_dtype) || !float_type(d->sum_dtype) || !float_type(d->weight_dtype) || !float_type(d->grad_dtype))
    return gtp::fail(GTP_E_DTYPE, "dtypes must be F32 or BF16");
  if (d->rows < 0 || d->cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (d->rows > kMaxRows || d->cols > kMaxCols) return gtp::fail(GTP_E_SHAPE, "rows above 2^30 or cols above 16384");
  if (d->grad_offset < 0 || d->grad_numel_total < 0 || d->grad_numel_total > (int64_t(1) << 50) ||
      d->grad_offset > d->grad_numel_total || d->cols > d->grad_numel_total - d->grad_offset)
    return gtp::fail(GTP_E_RANGE, "the view of %lld elements at %lld leaves a buffer of %lld", (long long)d->cols,
                     (long long)d->grad_offset, (long long)d->grad_numel_total);
  if (d->rows == 0 || d->cols == 0) return GTP_OK;
  const int64_t R = d->rows, C = d->cols;
  const Matrix dy = {"dy", d->dy, d->dy_ld, d->dy_dtype}, s = {"sum", d->sum, d->sum_ld, d->sum_dtype},
               ds = {"dsum", d->dsum, d->dsum_ld, d->sum_dtype}, dx = {"dx", d->dx, d->dx_ld, d->sum_dtype},
               w = {"weight", d->weight, C, d->weight_dtype};
  for (const Matrix *m : {&dy, &s, &dx})
    if (gtp_status e = check_matrix(*m, R, C)) return e;
  if (gtp_status e = check_matrix(w, 1, C)) return e;
  if (d->dsum)
    if (gtp_status e = check_matrix(ds, R, C)) return e;
  if (!d->rstd || !d->grad_data || !workspace) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t gs = size_of(d->grad_dtype);
  if (!aligned(d->rstd, 4) || !aligned(d->grad_data, gs) || !aligned(workspace, 16))
    return gtp::fail(GTP_E_ALIGN, "rstd and grad_data must be aligned to their elements, the workspace to 16 bytes");
  const int64_t need = gtp_rmsnorm_grad_workspace_bytes(R, C);
  if (workspace_bytes < need)
    return gtp::fail(GTP_E_CAPACITY, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
  char *const grad = static_cast<char *>(d->grad_data) + d->grad_offset * gs;
  const gtp::Runs out[3] = {runs_of(dx, R, C), runs_of(grad, C * gs), runs_of(workspace, need)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (gtp::overlap(out[i], out[j])) return gtp::fail(GTP_E_ARG, "dx, the gradient view and the workspace overlap");
    const gtp::Runs in[4] = {runs_of(dy, R, C), runs_of(s, R, C), runs_of(w, 1, C), runs_of(d->rstd, 4 * R)};
    const bool fine[4] = {i == 0 && same_place(dx, dy, R), i == 0 && same_place(dx, s, R), false, false};
    for (int j = 0; j < 4; ++j)
      if (!fine[j] && gtp::overlap(out[i], in[j])) return gtp::fail(GTP_E_ARG, "an output overlaps an input and is not it");
    if (d->dsum && !(i == 0 && same_place(dx, ds, R)) && gtp::overlap(out[i], runs_of(ds, R, C)))
      return gtp::fail(GTP_E_ARG, "an output overlaps dsum and is not it");
  }
  bool vec = C % 8 == 0 && vector_rows(dy, R) && vector_rows(s, R) && vector_rows(dx, R) && aligned(w.p, 16);
  if (d->dsum) vec = vec && vector_rows(ds, R);
  gtp::DeviceInfo dev;
  if (gtp_status e = gtp::require_sm103(&dev)) return e;
  GradArgs a = {};
  a.dy = d->dy, a.sum = d->sum, a.weight = d->weight, a.dsum = d->dsum, a.rstd = d->rstd, a.dx = d->dx;
  a.part = static_cast<float *>(workspace);
  a.rows = R, a.cols = C;
  a.dy_ld = R > 1 ? d->dy_ld : C, a.sum_ld = R > 1 ? d->sum_ld : C;
  a.dsum_ld = R > 1 ? d->dsum_ld : C, a.dx_ld = R > 1 ? d->dx_ld : C;
  a.weight_f32 = d->weight_dtype == GTP_F32;
  const GradShape shape = grad_shape(R, C, std::min(dev.sm_count, kMostSms));
  cudaStream_t st = gtp::as_stream(stream);
  using B = __nv_bfloat16;
  gtp_status e;
  if (d->dy_dtype == GTP_F32)
    e = d->sum_dtype == GTP_F32 ? launch_grad<float, float>(a, vec, shape, st) : launch_grad<float, B>(a, vec, shape, st);
  else
    e = d->sum_dtype == GTP_F32 ? launch_grad<B, float>(a, vec, shape, st) : launch_grad<B, B>(a, vec, shape, st);
  if (e) return e;
  const unsigned grid = unsigned((C + 31) / 32);
  const int parts = shape.grid * shape.row.ty;
  if (d->grad_dtype == GTP_F32)
    return gtp::launch_overlapped(norm_weight_kernel<float>, grid, dim3(32, 32), 0, st, "rmsnorm_grad",
                                  static_cast<const float *>(a.part), parts, C, reinterpret_cast<float *>(grad));
  return gtp::launch_overlapped(norm_weight_kernel<B>, grid, dim3(32, 32), 0, st, "rmsnorm_grad",
                                static_cast<const float *>(a.part), parts, C, reinterpret_cast<B *>(grad));
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
  const int64_t items = rows * (cols / 8), words = tiled_scales ? (cols / 32 + 3) / 4 : 0;
  const unsigned grid = unsigned(std::min<int64_t>((items + 255) / 256, int64_t(dev.sm_count) * 16));
  cudaStream_t st = gtp::as_stream(stream);
  const int vec = aligned(out, 16);
  if (out_dt == GTP_F32)
    return gtp::launch_overlapped(mxfp8_dequantize_kernel<float>, grid, 256, 0, st, "mxfp8_dequantize", e4m3, e8m0, rows, cols,
                                  words, static_cast<float *>(out), vec);
  return gtp::launch_overlapped(mxfp8_dequantize_kernel<__nv_bfloat16>, grid, 256, 0, st, "mxfp8_dequantize", e4m3, e8m0, rows,
                                cols, words, static_cast<__nv_bfloat16 *>(out), vec);
}
