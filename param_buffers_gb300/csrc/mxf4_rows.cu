// The MXFP4 forward and dgrad of a few rows (single tokens): D = dq(A) dq(B)^T, A of at most 4 rows.
//
// Page: "01 · ColumnParallelLinear / RowParallelLinear and the core autograd" (llm-infra-atlas), §4.1, §4.2,
// on the views of mxfp4.cu.
//
// The matrix B is read once and the tokens are nothing beside it, so the kernel is a reader: a lane takes one
// block of 32 codes (16 bytes, one scale) of four rows of B, all in flight together, and the warps of a
// block split the contraction until a lane has one such step.  The four rows are 32 apart, because the scale
// bytes of rows r, r + 32, r + 64, r + 96 under four blocks are the 16 bytes that four lanes read as one.
//
// A block's sum of products is exact: E2M1 values are multiples of 1/2 up to 6, so eight products in an fp16
// lane reach 288 in steps of 1/4, within its 11 bits; four such lanes are added in fp32, scaled by the
// blocks' powers of two and added up, lanes and warps in a fixed order.
//
// Measured, one token (two, four; the tensor-core kernel, whose time hardly depends on them), B of
//   [8192, 2048]    4.6 us  (6.6,  7.9;  7.2 - 7.5)   [8192, 4096]    6.8  (10.1, 13.4;  9.7 - 11.7)
//   [2048, 8192]    4.5     (6.6,  7.9; 12.3)         [4096, 16384]  10.0  (14.5, 21.5; 21 - 24)
//   [2048, 4096]    4.0     (4.8,  4.8;  8.1)         [28672, 8192]  31.3  (48.3, 77;   37 - 39)
//   [1536, 2048]    2.8     (3.8,  4.3;  5.4)         [8192, 28672]  27.5  (39.8, 65.6; 52 - 57)
//   [2048, 1024]    2.5     (3.1,  3.7;  4.4)         [64128, 2048]  19.0  (28.5, 44.7; 21 - 23)
//                                                     [128256, 2048] 35.1  (52.9, 87;   35)
// About 2.5 us of each is launch, first loads and the way out.  On large matrices it runs at 3.9 - 4.6 TB/s of the
// copy's 6.8: blocks come and go, and while one multiplies and adds up its sums it loads nothing.  A persistent form
// with a ring of asynchronous copies 100 KB an SM deep is bound by instructions instead (73 % of the issue
// slots; 26.3 us on [28672, 8192]) and costs the small matrices 0.5 - 1 us; the same loads feeding legacy 16-bit matrix
// instructions cost more in unpacking to bf16 than they saved (6.5 us on [8192, 2048], 15 on
// [2048, 8192]); asking for B's lines in L2 before the previous kernel ends gave 0.1 us; unpacking by shifts and
// masks instead of the conversion takes 5.5 us on [8192, 2048].
//
// Hence the rule in few_rows(): one token always; up to four while they and B's rows are few, where the tensor-core
// kernel's tiles of 256 columns leave SMs idle and each waits for its own chain of loads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "mxf4_rows.h"
#include "sm100_ptx.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kGroupRows = 4;  // rows of B a warp holds
// A block's sum (below 2^11) is scaled by the token's power of two, times this, and then by the row's: the first
// product neither overflows nor loses a bit under any scale byte, the second only where the result does.
constexpr float kShift = 0x1p-16f;

struct RowsArgs {
  const uint8_t *a, *as, *b, *bs;
  __nv_bfloat16 *d;
  int64_t n_dim, blocks, words;  // rows of B; blocks of a row; scale atoms of a row tile
  int32_t m_dim, k_warps;        // k_warps: the warps along the contraction, a power of two
};

// Eight codes to four half pairs; exact.
__device__ __forceinline__ void halves(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ void block_halves(const uint4 &c, uint32_t (&h)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t q[4];
    halves(w[i], q);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[4 * i + j] = q[j];
  }
}

__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }

__device__ __forceinline__ float block_dot(const uint32_t (&x)[16], const uint32_t (&y)[16]) {
  __half2 s0 = __hmul2(half2_of(x[0]), half2_of(y[0])), s1 = __hmul2(half2_of(x[8]), half2_of(y[8]));
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    s0 = __hfma2(half2_of(x[i]), half2_of(y[i]), s0);
    s1 = __hfma2(half2_of(x[8 + i]), half2_of(y[8 + i]), s1);
  }
  // the four lanes' sums into fp32, each half taken as it lies
  float r;
  asm("{\n\t.reg .b16 a, b, c, d, one;\n\t.reg .f32 f;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 {c, d}, %2;\n\t"
      "mov.b16 one, 0x3C00;\n\tfma.rn.f32.f16 f, a, one, 0f00000000;\n\tfma.rn.f32.f16 f, b, one, f;\n\t"
      "fma.rn.f32.f16 f, c, one, f;\n\tfma.rn.f32.f16 %0, d, one, f;\n\t}"
      : "=f"(r)
      : "r"(*reinterpret_cast<const uint32_t *>(&s0)), "r"(*reinterpret_cast<const uint32_t *>(&s1)));
  return r;
}

// 2^(byte - 127), NaN for 0xFF.
__device__ __forceinline__ float scale_f32(uint32_t byte) {
  return __uint_as_float(byte == 0xFFu ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// Blocks an SM by the tokens held: what the registers allow without (or nearly without) spilling.
template <int MT>
constexpr int kMinBlocks = MT == 1 ? 4 : MT == 2 ? 3 : 2;

template <int MT>
__global__ void __launch_bounds__(32 * kWarps, kMinBlocks<MT>) mx4_rows_kernel(const __grid_constant__ RowsArgs p) {
  constexpr int V = MT * kGroupRows;
  __shared__ float partial[kWarps][V];
  gtp::ptx::allow_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = kWarps / p.k_warps;
  const int kw = warp & (p.k_warps - 1), g = warp / p.k_warps;
  const int64_t group = int64_t(blockIdx.x) * groups + g, tile = group >> 5;
  const int r0 = int(group & 31);
  const int64_t n0 = 128 * tile + r0;
  gtp::ptx::wait_prior_grid();
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  if (n0 < p.n_dim) {
    for (int64_t k = 32 * kw + lane; k < p.blocks; k += 32 * p.k_warps) {
      uint4 c[kGroupRows];
#pragma unroll
      for (int i = 0; i < kGroupRows; ++i) {
        c[i] = make_uint4(0, 0, 0, 0);
        if (n0 + 32 * i < p.n_dim)
          c[i] = *(reinterpret_cast<const uint4 *>(p.b) + (n0 + 32 * i) * p.blocks + k);
      }
      const uint4 s = *(reinterpret_cast<const uint4 *>(p.bs + (tile * p.words + (k >> 2)) * 512) + r0);
      uint4 x[MT];
      uint32_t sx[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        x[m] = make_uint4(0, 0, 0, 0);
        sx[m] = 0;
        if (m < p.m_dim) {
          x[m] = *(reinterpret_cast<const uint4 *>(p.a) + m * p.blocks + k);
          sx[m] = p.as[(k >> 2) * 512 + 16 * m + (k & 3)];
        }
      }
      const uint32_t sw[kGroupRows] = {s.x, s.y, s.z, s.w};
      float fx[MT], fw[kGroupRows];
      uint32_t xh[MT][16];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        fx[m] = kShift * scale_f32(sx[m]);
        block_halves(x[m], xh[m]);
      }
#pragma unroll
      for (int i = 0; i < kGroupRows; ++i) fw[i] = scale_f32((sw[i] >> (8 * (lane & 3))) & 0xFFu);
#pragma unroll
      for (int i = 0; i < kGroupRows; ++i) {
        uint32_t h[16];
        block_halves(c[i], h);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[kGroupRows * m + i] += block_dot(xh[m], h) * fx[m] * fw[i];
      }
    }
  }
  // over the lanes: halving the values a lane holds while there are several, then plain sums
  int w = 16;
#pragma unroll
  for (int n = V; n > 1; n >>= 1, w >>= 1) {
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) {
      const float mine = upper ? acc[j + n / 2] : acc[j], theirs = upper ? acc[j] : acc[j + n / 2];
      acc[j] = mine + __shfl_xor_sync(0xFFFFFFFFu, theirs, w);
    }
  }
  for (; w; w >>= 1) acc[0] += __shfl_xor_sync(0xFFFFFFFFu, acc[0], w);
  if ((lane & (32 / V - 1)) == 0) partial[warp][lane / (32 / V)] = acc[0];
  __syncthreads();
  // over the warps of a group, and out
  if (int(threadIdx.x) < groups * V) {
    const int q = threadIdx.x / V, v = threadIdx.x % V, m = v / kGroupRows;
    const int64_t to = int64_t(blockIdx.x) * groups + q, n = 128 * (to >> 5) + (to & 31) + 32 * (v % kGroupRows);
    float sum = 0.f;
    for (int i = 0; i < p.k_warps; ++i) sum += partial[q * p.k_warps + i][v];
    if (m < p.m_dim && n < p.n_dim) p.d[m * p.n_dim + n] = __float2bfloat16_rn(sum / kShift);
  }
}

}  // namespace

namespace gtp {

bool few_rows(int64_t m_dim, int64_t n_dim, int sm_count) {
  return m_dim == 1 || (m_dim <= 4 && m_dim * n_dim <= 128 * int64_t(sm_count));
}

gtp_status run_mxfp4_rows(const uint8_t *Aq, const uint8_t *As, const uint8_t *Bq, const uint8_t *Bs, void *D,
                          int64_t m_dim, int64_t n_dim, int64_t k_dim, cudaStream_t st) {
  RowsArgs p = {};
  p.a = Aq, p.as = As, p.b = Bq, p.bs = Bs;
  p.d = static_cast<__nv_bfloat16 *>(D);
  p.n_dim = n_dim;
  p.blocks = (k_dim + 31) / 32;
  p.words = (p.blocks + 3) / 4;
  p.m_dim = int32_t(m_dim);
  p.k_warps = 1;
  // as many as leave every lane a step: the fewest steps in a row, and the most loads in flight
  while (p.k_warps < kWarps && 32 * p.k_warps < p.blocks) p.k_warps *= 2;
  const int64_t row_groups = (n_dim + 127) / 128 * 32, per_block = kWarps / p.k_warps;
  const dim3 grid(unsigned((row_groups + per_block - 1) / per_block)), block(32 * kWarps);
  if (m_dim == 1) return launch_overlapped(mx4_rows_kernel<1>, grid, block, 0, st, "mxfp4_rows", p);
  if (m_dim == 2) return launch_overlapped(mx4_rows_kernel<2>, grid, block, 0, st, "mxfp4_rows", p);
  return launch_overlapped(mx4_rows_kernel<4>, grid, block, 0, st, "mxfp4_rows", p);
}

}  // namespace gtp
