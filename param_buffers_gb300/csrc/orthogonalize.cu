// The orthogonalised update of the layer-wise optimizer: Newton-Schulz products on the 5th-generation tensor cores, and
// the whole step on weights of the flat buffers.
//
// Page: "05 · grad/param buffer ..." (llm-infra-atlas), §3 and §6.5 (parameters managed by a layer-wise optimizer have
// buffers of their own; the optimizer reads main_grad and writes the master and the parameter).  The rule is that of
// Jordan et al., "Muon: an optimizer for hidden layers in neural networks", 2024 (momentum, Nesterov, the quintic
// iteration and its coefficients).
//
//   X = G / |G|_F;   steps times:   A = X X^T,  B = b A + c A^2,  X <- a X + B X
// with the smaller Gram matrix: for more rows than columns A = X^T X and X <- a X + X B.
//
// Three products an iteration, each one launch of a CTA-pair kernel.  A and A^2 are symmetric: only tiles on and above
// the diagonal are computed, each is written twice.
//
// Precision.  The operands are fp16, whose 11 bits err an eighth of bf16's at the same rate; all values here are bounded
// (|X|_2 stays near 1), so powers of two hold them in fp16's range.  Three choices keep rounding away from where the
// polynomial's terms cancel (a + b + c = 0.7 out of terms up to 4.8):
//   - the diagonals of A and B never become fp16: d = diag(A) and e = a + diag(B) stay fp32 vectors, with A = d + A'
//     the square is d^2 + (d_i + d_j) A' + A'^2, and X <- e X + B' X;
//   - the X of the linear term is fp16 high part + fp16 low part (22 bits); the products read the high part alone.  The
//     low part is scaled by e where X is nearly orthogonal (B' is small there: what its product leaves out is small),
//     but by a alone in the first two iterations, where small singular values, on which a + diag(B) acts as far more
//     than a + B does, still grow threefold each;
//   - A' enters B' with a low part of its own (the square reads the high part).
// Against fp64, relative error of the result: 2e-4 to 1e-3 over Gaussian, row-scaled and low-rank matrices; without the
// first two 2e-3 to 9e-3, with bf16 operands 1.4e-2 to 6e-2.  A bf16 result's own rounding is 1.7e-3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "byte_range.h"
#include "device.h"
#include "fastdiv.cuh"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace gtp {
void clear_error();
}

namespace {

using namespace gtp::ptx;

__device__ unsigned int g_ortho_wait_timeouts;  // this unit's part of gtp_wait_timeouts' word

constexpr int kMostMatrices = 64;

// --------------------------------------------------------------------------- the norm, the momentum, the first X

struct Source {
  const void *src;  // [count] planes of [rows, cols], or (src null) the momentum's update
  int64_t ld, plane;
  // the step: u = mu m' + (1 - mu) g where m' = mu m + (1 - mu) g, or u = m'
  void *grad;
  float *momentum;
  int64_t offset[kMostMatrices];
  const float *grad_scale;
  float mu, factor;
  int nesterov, zero_grad;
  int rows, cols;
  gtp::FastDiv by_cols;  // cols / 4 with VEC, else cols
  int items;             // of a matrix
};

struct FirstX {
  double *part;  // [count][gridDim.x]: sums of squares
  __half *hi, *lo, *hi_next;
  int64_t ldx, planex;
  float xscale;
  int parts, rows;  // rows: of X, those behind the matrix's zero
};

__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// The elements of item i of matrix k (four consecutive ones of a row with VEC, else one): the matrix's own, or the
// step's u.  FIRST: the pass that writes the momentum; the second finds it written and clears the gradient.
template <typename T, bool VEC, bool STEP, bool FIRST>
__device__ __forceinline__ void source_at(const Source &s, int k, int i, float g_scale, int &row, int &col,
                                          float (&x)[VEC ? 4 : 1]) {
  constexpr int E = VEC ? 4 : 1;
  row = gtp::fast_div(i, s.by_cols);
  col = (i - row * (s.cols / E)) * E;
  if (!STEP) {
    const T *p = static_cast<const T *>(s.src) + k * s.plane + row * s.ld + col;
    if constexpr (VEC) load4(p, x);
    else x[0] = load1(p);
    return;
  }
  const int64_t at = s.offset[k] + int64_t(row) * s.cols + col;
  T *const gp = static_cast<T *>(s.grad) + at;
  float *const mp = s.momentum + at;
  float g[E], m[E];
  if constexpr (VEC) {
    load4(gp, g);
    load4(mp, m);
  } else {
    g[0] = load1(gp);
    m[0] = *mp;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    g[e] *= g_scale;
    if (FIRST) m[e] = fmaf(s.mu, m[e], (1.f - s.mu) * g[e]);
    x[e] = s.nesterov ? fmaf(s.mu, m[e], (1.f - s.mu) * g[e]) : m[e];
  }
  if (FIRST) {
    if constexpr (VEC) *reinterpret_cast<float4 *>(mp) = make_float4(m[0], m[1], m[2], m[3]);
    else *mp = m[0];
  } else if (s.zero_grad) {
    if constexpr (!VEC) gp[0] = T(0.f);
    else if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(gp) = make_float4(0.f, 0.f, 0.f, 0.f);
    else *reinterpret_cast<uint2 *>(gp) = make_uint2(0u, 0u);
  }
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double sums[32];
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < int(blockDim.x >> 5); ++w) v += sums[w];
  return v;
}

constexpr int kPassThreads = 256;

// Sums of squares, a block's part each (and the new momentum).
template <typename T, bool VEC, bool STEP>
__global__ void __launch_bounds__(kPassThreads)
    squares_kernel(const __grid_constant__ Source s, const __grid_constant__ FirstX f) {
  allow_dependents();
  wait_prior_grid();
  const float g_scale = STEP ? s.factor * (s.grad_scale ? *s.grad_scale : 1.f) : 1.f;
  double total = 0;
  for (int64_t i0 = int64_t(blockIdx.x) * kPassThreads; i0 < s.items; i0 += 4 * int64_t(gridDim.x) * kPassThreads) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + int64_t(j) * gridDim.x * kPassThreads + threadIdx.x;
      if (i < s.items) {
        int row, col;
        float x[VEC ? 4 : 1];
        source_at<T, VEC, STEP, true>(s, blockIdx.y, int(i), g_scale, row, col, x);
#pragma unroll
        for (int e = 0; e < (VEC ? 4 : 1); ++e) sum = fmaf(x[e], x[e], sum);
      }
    }
    total += double(sum);
  }
  total = block_sum(total);
  if (threadIdx.x == 0) f.part[blockIdx.y * gridDim.x + blockIdx.x] = total;
}

// X = G / |G|_F as fp16 high and low parts, times a power of two.  A matrix of zeros stays zero; one whose squares'
// sum is not finite becomes NaN.
template <typename T, bool VEC, bool STEP>
__global__ void __launch_bounds__(kPassThreads)
    first_x_kernel(const __grid_constant__ Source s, const __grid_constant__ FirstX f) {
  allow_dependents();
  wait_prior_grid();
  const float g_scale = STEP ? s.factor * (s.grad_scale ? *s.grad_scale : 1.f) : 1.f;
  double total = 0;
  for (int p = threadIdx.x; p < f.parts; p += kPassThreads) total += f.part[blockIdx.y * f.parts + p];
  total = block_sum(total);
  const float r = total == 0 ? 0.f : isfinite(total) ? float(double(f.xscale) / sqrt(total)) : nanf("");
  const int step = int(gridDim.x) * kPassThreads, me = int(blockIdx.x) * kPassThreads + int(threadIdx.x);
  const int64_t zeros = (f.rows - s.rows) * f.ldx / 8;  // in both buffers that take turns as the products' X
  for (int64_t i = me; i < zeros; i += step) {
    const int64_t at = blockIdx.y * f.planex + s.rows * f.ldx + 8 * i;
    *reinterpret_cast<uint4 *>(f.hi + at) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4 *>(f.hi_next + at) = make_uint4(0, 0, 0, 0);
  }
  for (int64_t i = me; i < s.items; i += step) {
    int row, col;
    float x[VEC ? 4 : 1];
    source_at<T, VEC, STEP, false>(s, blockIdx.y, int(i), g_scale, row, col, x);
    const int64_t at = blockIdx.y * f.planex + row * f.ldx + col;
    __half hi[VEC ? 4 : 1], lo[VEC ? 4 : 1];
#pragma unroll
    for (int e = 0; e < (VEC ? 4 : 1); ++e) {
      const float v = x[e] * r;
      hi[e] = __float2half_rn(v);
      lo[e] = __float2half_rn(v - __half2float(hi[e]));
    }
    if constexpr (VEC) {
      *reinterpret_cast<uint2 *>(f.hi + at) = *reinterpret_cast<const uint2 *>(hi);
      *reinterpret_cast<uint2 *>(f.lo + at) = *reinterpret_cast<const uint2 *>(lo);
    } else {
      f.hi[at] = hi[0];
      f.lo[at] = lo[0];
    }
  }
}

// --------------------------------------------------------------------------- the products

constexpr int BK = 64, UK = 16, BMC = 128, BMP = 256;
constexpr int A_STAGE = BMC * BK * 2;
constexpr int MN_CHUNK = 64 * BK * 2;  // one 64-wide MN-major box
constexpr int SMEM_OPS = 192 * 1024, SMEM_CTRL = 512;
constexpr int SMEM_TOTAL = SMEM_OPS + SMEM_CTRL + 1024;
// warps: 0 A producer, 1 MMA, 2 B producer, 4-11 epilogue (two a quarter of the accumulator's lanes)
constexpr int kThreads = 384, kEpilogueWarps = 8;

template <int BN>
struct Ring {
  static constexpr int B_STAGE = BN / 2 * BK * 2;
  static constexpr int STAGE = A_STAGE + B_STAGE;
  static constexpr int STAGES = SMEM_OPS / STAGE;
};

enum Epilogue { kGram, kPoly, kUpdate, kOut, kStep };

struct Product {
  int tiles_m, tiles_n, k_blocks;
  int each, units;       // units of a matrix, of all
  int a_rows, b_rows;    // a matrix's rows in either operand
  int symmetric, n_fast; // tiles on and above the diagonal only; which index of the tiles runs first
  int m_dim, n_dim;      // of the output
  // kGram, kPoly
  __half *gram, *gram_lo, *poly;  // A' (high and low part) and B'
  int64_t ldg, planeg;
  float *diag, *e;       // [count][m]
  int m;
  // kUpdate and the last product
  const __half *hi;
  __half *hi_out, *lo;
  int64_t ldx, planex;
  int tall, early;       // early: one of the first two iterations
  // powers of two: what makes the accumulator, A', B' and X true values and the reverse
  float alpha, gram_scale, gram_inv, poly_scale, x_scale, x_inv;
  float a, b, c;
  // kOut
  void *dst;
  int64_t ld, plane;
  int dst_f32;
  // kStep
  float *master;
  __nv_bfloat16 *param;
  float keep, rate;      // 1 - lr wd, lr scale
  int64_t offset[kMostMatrices];
};

template <int BN>
__device__ __forceinline__ void decode(const Product &p, int u, int &k, int &tm, int &tn) {
  k = u / p.each;
  int t = u - k * p.each;
  if (p.symmetric) {
    tm = 0;
    for (;;) {
      tn = tm * (BMP / BN);
      const int n = p.tiles_n - tn;
      if (t < n) break;
      t -= n;
      ++tm;
    }
    tn += t;
  } else if (p.n_fast) {
    tm = t / p.tiles_n;
    tn = t - tm * p.tiles_n;
  } else {
    tn = t / p.tiles_m;
    tm = t - tn * p.tiles_m;
  }
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((7u << 7) | (7u << 10));  // formats 0: fp16
}

__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(&g_ortho_wait_timeouts, 0x80u);
      return;
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// 32 fp16 of one row, on 64 bytes.
__device__ __forceinline__ void load_row(const __half *p, uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 v = reinterpret_cast<const uint4 *>(p)[q];
    w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
  }
}
__device__ __forceinline__ void store_row(__half *p, const uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    reinterpret_cast<uint4 *>(p)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}

// A row's 32 fp16 of a symmetric matrix, and the same below the diagonal where no tile computes them.
__device__ __forceinline__ void store_symmetric(__half *out, int64_t ld, int m, int row, int col, const uint32_t (&w)[16]) {
  store_row(out + row * ld + col, w);
  if (col / BMP > row / BMP) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col + j < m)
        reinterpret_cast<uint16_t *>(out)[(col + j) * ld + row] = uint16_t(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
  }
}

// What becomes of 32 columns of one row of the accumulator.
template <int EPI>
__device__ __forceinline__ void finish(const Product &p, int k, int row, int col, const uint32_t (&acc)[32]) {
  if (row >= p.m_dim || col >= p.n_dim) return;
  if constexpr (EPI == kGram || EPI == kPoly) {
    uint32_t w[16], g[16], l[16];
    float di = 0.f;
    const float *const d = p.diag + int64_t(k) * p.m;
    __half *const gram = p.gram + k * p.planeg, *const gram_lo = p.gram_lo + k * p.planeg;
    if (EPI == kPoly) {
      load_row(gram + row * p.ldg + col, g);
      load_row(gram_lo + row * p.ldg + col, l);
      di = d[row];
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float v[2];
      const float2 old = EPI == kPoly ? unpack2(g[j >> 1]) : make_float2(0.f, 0.f);
      const float2 low = EPI == kPoly ? unpack2(l[j >> 1]) : make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float s = __uint_as_float(acc[j + i]) * p.alpha;
        const bool on_diagonal = col + j + i == row;
        if (EPI == kGram) {
          if (on_diagonal) p.diag[int64_t(k) * p.m + row] = s;
          v[i] = on_diagonal ? 0.f : s * p.gram_scale;
        } else {
          if (on_diagonal) p.e[int64_t(k) * p.m + row] = fmaf(p.c, fmaf(di, di, s), fmaf(p.b, di, p.a));
          const float dj = col + j + i < p.m ? d[col + j + i] : 0.f;
          const float a = (i ? old.y + low.y : old.x + low.x) * p.gram_inv;
          v[i] = on_diagonal ? 0.f : (p.b * a + p.c * fmaf(di + dj, a, s)) * p.poly_scale;
        }
      }
      w[j >> 1] = pack2(v[0], v[1]);
      if (EPI == kGram) {
        const float2 high = unpack2(w[j >> 1]);
        l[j >> 1] = pack2(v[0] - high.x, v[1] - high.y);
      }
    }
    if (EPI == kGram) store_row(gram_lo + row * p.ldg + col, l);  // where kPoly's own tiles are
    store_symmetric(EPI == kGram ? gram : p.poly + k * p.planeg, p.ldg, p.m, row, col, w);
  } else {
    const int64_t at = k * p.planex + row * p.ldx + col;
    uint32_t h[16], l[16];
    load_row(p.hi + at, h);
    load_row(p.lo + at, l);
    float x[32];
    const float *const e = p.e + int64_t(k) * p.m;
    const float er = p.tall ? 0.f : e[row];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 a = unpack2(h[j >> 1]), b = unpack2(l[j >> 1]);
      const float e0 = p.tall ? (col + j < p.m ? e[col + j] : 0.f) : er;
      const float e1 = p.tall ? (col + j + 1 < p.m ? e[col + j + 1] : 0.f) : er;
      // x_inv times the stored X, alpha times the accumulator: true values
      const float x0 = p.early ? fmaf(e0, a.x, p.a * b.x) : e0 * (a.x + b.x);
      const float x1 = p.early ? fmaf(e1, a.y, p.a * b.y) : e1 * (a.y + b.y);
      x[j] = fmaf(x0, p.x_inv, __uint_as_float(acc[j]) * p.alpha);
      x[j + 1] = fmaf(x1, p.x_inv, __uint_as_float(acc[j + 1]) * p.alpha);
    }
    if constexpr (EPI == kUpdate) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float x0 = x[j] * p.x_scale, x1 = x[j + 1] * p.x_scale;
        h[j >> 1] = pack2(x0, x1);
        const float2 r = unpack2(h[j >> 1]);
        l[j >> 1] = pack2(x0 - r.x, x1 - r.y);
      }
      store_row(p.hi_out + at, h);
      store_row(p.lo + at, l);
    } else if constexpr (EPI == kOut) {
      const int n = min(32, p.n_dim - col);
      const int64_t to = k * p.plane + row * p.ld + col;
      if (p.dst_f32) {
        float *const o = static_cast<float *>(p.dst) + to;
        if (n == 32 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            reinterpret_cast<float4 *>(o)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < n) o[j] = x[j];
        }
      } else {
        __nv_bfloat16 *const o = static_cast<__nv_bfloat16 *>(p.dst) + to;
        __nv_bfloat162 w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        if (n == 32 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) reinterpret_cast<uint4 *>(o)[q] = reinterpret_cast<const uint4 *>(w)[q];
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < n) o[j] = j & 1 ? __high2bfloat16(w[j >> 1]) : __low2bfloat16(w[j >> 1]);
        }
      }
    } else {
      const int n = min(32, p.n_dim - col);
      const int64_t to = p.offset[k] + int64_t(row) * p.n_dim + col;
      float *const o = p.master + to;
      const bool wide = n == 32 && (reinterpret_cast<uintptr_t>(o) & 15) == 0;
      if (wide) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 v = reinterpret_cast<const float4 *>(o)[q];
          x[4 * q] = fmaf(p.keep, v.x, -p.rate * x[4 * q]);
          x[4 * q + 1] = fmaf(p.keep, v.y, -p.rate * x[4 * q + 1]);
          x[4 * q + 2] = fmaf(p.keep, v.z, -p.rate * x[4 * q + 2]);
          x[4 * q + 3] = fmaf(p.keep, v.w, -p.rate * x[4 * q + 3]);
          reinterpret_cast<float4 *>(o)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n) {
            x[j] = fmaf(p.keep, o[j], -p.rate * x[j]);
            o[j] = x[j];
          }
      }
      if (p.param) {
        __nv_bfloat16 *const q = p.param + to;
        __nv_bfloat162 w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        if (wide && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) reinterpret_cast<uint4 *>(q)[i] = reinterpret_cast<const uint4 *>(w)[i];
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < n) q[j] = j & 1 ? __high2bfloat16(w[j >> 1]) : __low2bfloat16(w[j >> 1]);
        }
      }
    }
  }
}

// D = A B^T of one pair tile of 256 x BN after another, over a CTA pair (a cluster of two SMs sharing M = 256 MMAs):
// each CTA stages 128 rows of A and BN / 2 rows of B a k-block and holds its 128 x BN of D in tensor memory, twice, so
// that a tile's epilogue runs under the next one's products.  The hand-offs are those of the bf16 pair GEMM: both CTAs'
// copies complete on the even CTA's full[], which that CTA arms; its commits go to both CTAs' empty[] and tfull[]; the
// epilogue warps of both release an accumulator on its tempty[]; at exit it drains every stage that it armed.
template <int BN, bool A_MN, bool B_MN, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    newton_schulz_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ Product p) {
  using R = Ring<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sA = smem, *sB = smem + R::STAGES * A_STAGE;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + SMEM_OPS);
  uint64_t *empty = full + R::STAGES;
  uint64_t *tfull = empty + R::STAGES;
  uint64_t *tempty = tfull + 2;
  uint64_t *drained = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert((2 * R::STAGES + 5) * 8 + 8 <= SMEM_CTRL, "control block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int first = int(blockIdx.x >> 1), step = int(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < R::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpilogueWarps);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrive or multicast
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  unsigned int *err = &g_ortho_wait_timeouts;
  allow_dependents();
  wait_prior_grid();

  if (warp == 0) {
    if (lane == 0) {  // -------------------------------------------------- A producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      int armed[R::STAGES];
      for (int s = 0; s < R::STAGES; ++s) armed[s] = -1;
      bool ok = true;
      for (int u = first; ok && u < p.units; u += step) {
        int k, tm, tn;
        decode<BN>(p, u, k, tm, tn);
        const int m0 = tm * BMP + BMC * int(rank);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err, 0x1u)) {
            ok = false;
            break;
          }
          if (rank == 0) {
            mbar_arrive_expect_tx(&full[stage], 2u * uint32_t(R::STAGE));
            armed[stage] = int(phase);
          }
          const uint32_t bar = mapa_shared(&full[stage], 0);
          uint8_t *a = sA + stage * A_STAGE;
          if (A_MN) {
            tma_load_2d_pair(&tmA, bar, a, m0, k * p.a_rows + kb * BK);
            tma_load_2d_pair(&tmA, bar, a + MN_CHUNK, m0 + 64, k * p.a_rows + kb * BK);
          } else {
            tma_load_2d_pair(&tmA, bar, a, kb * BK, k * p.a_rows + m0);
          }
          if (++stage == R::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      for (int s = 0; s < R::STAGES; ++s)
        if (armed[s] >= 0) drain(&full[s], uint32_t(armed[s]));
    }
  } else if (warp == 2) {
    if (lane == 0) {  // -------------------------------------------------- B producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; ok && u < p.units; u += step) {
        int k, tm, tn;
        decode<BN>(p, u, k, tm, tn);
        const int n0 = tn * BN + (BN / 2) * int(rank);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err, 0x1u)) {
            ok = false;
            break;
          }
          const uint32_t bar = mapa_shared(&full[stage], 0);
          uint8_t *b = sB + stage * R::B_STAGE;
          if (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_2d_pair(&tmB, bar, b + j * MN_CHUNK, n0 + 64 * j, k * p.b_rows + kb * BK);
          } else {
            tma_load_2d_pair(&tmB, bar, b, kb * BK, k * p.b_rows + n0);
          }
          if (++stage == R::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {  // ---------------------------------------------- MMA (the even CTA)
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(BMP, BN, A_MN, B_MN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = first; ok && u < p.units; u += step) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, err, 0x2u))) break;
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc * BN);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, abort_flag, err, 0x4u))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one_sync()) {
            const uint32_t a0 = smem_u32(sA + stage * A_STAGE), b0 = smem_u32(sB + stage * R::B_STAGE);
#pragma unroll
            for (int i = 0; i < BK / UK; ++i) {
              const uint64_t ad = A_MN ? sdesc_sw128(a0 + i * (UK * 128), MN_CHUNK, 1024) : sdesc_sw128(a0 + i * (UK * 2), 16, 1024);
              const uint64_t bd = B_MN ? sdesc_sw128(b0 + i * (UK * 128), MN_CHUNK, 1024) : sdesc_sw128(b0 + i * (UK * 2), 16, 1024);
              mma_f16_pair(d, ad, bd, idesc, (kb > 0 || i > 0) ? 1u : 0u);
            }
            mma_commit_pair(&empty[stage], 0x3);
          }
          __syncwarp();
          if (++stage == R::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one_sync()) mma_commit_pair(&tfull[acc], 0x3);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (elect_one_sync()) mma_commit_pair(drained, 0x3);  // both CTAs learn when every MMA has finished
      __syncwarp();
    }
    if (lane == 0) drain(drained, 0);
  } else if (warp >= 4) {  // ---------------------------------------------- epilogue (both CTAs)
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < p.units; u += step) {
      int k, tm, tn;
      decode<BN>(p, u, k, tm, tn);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, abort_flag, err, 0x8u))) break;
      tc_fence_after();
      const int row = tm * BMP + BMC * int(rank) + 32 * quarter + lane;
      const int c0 = half * (BN / 2);
      const uint32_t base = tmem_base + (uint32_t(32 * quarter) << 16) + uint32_t(acc * BN + c0);
#pragma unroll 1
      for (int c = 0; c < BN / 2; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(base + uint32_t(c), r);
        tmem_ld_wait();
        finish<EPI>(p, k, row, tn * BN + c0 + c, r);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&tempty[acc], 0));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still reach its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * BN);
  }
}

// --------------------------------------------------------------------------- host

constexpr int64_t kMostElements = (int64_t(1) << 31) - 1, kMostSide = 65536;
constexpr int kMostSteps = 16, kMostParts = 256;

struct Plan {
  int64_t m, n, rows, ldx, planex, ldg, planeg;  // rows: of X with the zeros that fill a contraction's last block
  int64_t hi[2], lo, gram, gram_lo, poly, diag, e, part, bytes;  // places in the workspace
};

Plan plan_of(int64_t count, int64_t rows, int64_t cols) {
  Plan p = {};
  p.m = std::min(rows, cols), p.n = std::max(rows, cols);
  // whole 32-column chunks a row, whatever the matrix's own width: the epilogue needs no bounds inside a chunk, and
  // the copies stop at the true width
  p.rows = (rows + BK - 1) / BK * BK;
  p.ldx = (cols + 63) / 64 * 64, p.planex = p.rows * p.ldx;
  p.ldg = (p.m + 63) / 64 * 64, p.planeg = p.m * p.ldg;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) & ~int64_t(255);
    return here;
  };
  p.hi[0] = take(2 * count * p.planex);
  p.hi[1] = take(2 * count * p.planex);
  p.lo = take(2 * count * p.planex);
  p.gram = take(2 * count * p.planeg);
  p.gram_lo = take(2 * count * p.planeg);
  p.poly = take(2 * count * p.planeg);
  p.diag = take(4 * count * p.m);
  p.e = take(4 * count * p.m);
  p.part = take(8 * count * kMostParts);
  p.bytes = at;
  return p;
}

struct Schedule {
  float a, b, c;
  int steps;
  float bound;  // on |X|_2 over all iterations, from 1
};

// The largest singular value that the iteration can make of one in [0, 1], step by step, on a grid whose spacing the
// margin below covers; refused where it leaves what the fp16 scales hold.
gtp_status schedule_of(const float *abc, int32_t steps, Schedule *s) {
  if (!abc) return gtp::fail(GTP_E_ARG, "null coefficients");
  if (steps < 1 || steps > kMostSteps) return gtp::fail(GTP_E_ARG, "steps must be 1 to %d", kMostSteps);
  for (int i = 0; i < 3; ++i)
    if (!std::isfinite(abc[i]) || std::fabs(abc[i]) > 64.f) return gtp::fail(GTP_E_ARG, "coefficients must be finite, at most 64");
  const double a = abc[0], b = abc[1], c = abc[2];
  double top = 1.0, most = 1.0;
  for (int k = 0; k + 1 < steps; ++k) {  // the last result is the output, not an operand
    double next = 0;
    for (int i = 0; i <= 1024; ++i) {
      const double x = top * i / 1024, x2 = x * x;
      next = std::max(next, std::fabs(x * (a + b * x2 + c * x2 * x2)));
    }
    top = 1.01 * next;
    most = std::max(most, top);
    if (most > 2.0) return gtp::fail(GTP_E_ARG, "these coefficients let singular values grow past 2");
  }
  *s = {abc[0], abc[1], abc[2], steps, float(most)};
  return GTP_OK;
}

template <int BN, bool A_MN, bool B_MN, int EPI>
gtp_status launch_product(const CUtensorMap &ta, const CUtensorMap &tb, const Product &p, const gtp::DeviceInfo &dev,
                          cudaStream_t st) {
  static std::atomic<uint64_t> configured{0};
  const auto kernel = newton_schulz_kernel<BN, A_MN, B_MN, EPI>;
  const uint64_t bit = uint64_t(1) << (dev.device & 63);
  if (!(configured.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
    if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    configured.fetch_or(bit);
  }
  const unsigned grid = 2 * unsigned(std::min(p.units, dev.sm_count / 2));
  return gtp::launch_overlapped(kernel, grid, kThreads, SMEM_TOTAL, st, "orthogonalize", ta, tb, p);
}

// An operand: matrices of rows x inner fp16 at `base`, one after another.  A copy that passes a matrix's last row reads
// the next one's: harmless where rows are the product's rows or columns (nobody takes those), and where they are the
// contraction the last block's rows are zeros of the matrix's own (Plan::rows).
struct Operand {
  const void *base;
  int64_t inner, rows, ld;
};

gtp_status map_of(CUtensorMap *map, const Operand &o, int64_t count, bool mn, int box_rows) {
  return gtp::encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, o.base, uint64_t(o.inner), uint64_t(count * o.rows),
                             uint64_t(2 * o.ld), BK, mn ? 64 : uint32_t(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

// The product D = A B^T (m_dim x n_dim, contraction k) of every matrix, in tiles 256 columns wide or 128: whichever
// needs less time in whole waves of the machine's CTA pairs.  A half-wide tile takes 0.55 of a whole one's time.
template <bool A_MN, bool B_MN, int EPI>
gtp_status run_product(Product p, const Operand &a, const Operand &b, int64_t count, int64_t k, const gtp::DeviceInfo &dev,
                       cudaStream_t st) {
  const int pairs = dev.sm_count / 2;
  const auto shape = [&](int BN) {
    p.tiles_m = (p.m_dim + BMP - 1) / BMP;
    p.tiles_n = (p.n_dim + BN - 1) / BN;
    p.each = p.tiles_m * p.tiles_n;
    if (p.symmetric) {
      p.each = 0;
      for (int tm = 0; tm < p.tiles_m; ++tm) p.each += std::max(0, p.tiles_n - tm * (BMP / BN));
    }
    p.units = int(count) * p.each;
    return (p.units + pairs - 1) / pairs;
  };
  p.k_blocks = int((k + BK - 1) / BK);
  p.a_rows = int(a.rows), p.b_rows = int(b.rows);
  const bool narrow = 0.55 * shape(128) < shape(256);
  CUtensorMap ta, tb;
  if (gtp_status s = map_of(&ta, a, count, A_MN, BMC)) return s;
  if (gtp_status s = map_of(&tb, b, count, B_MN, narrow ? 64 : 128)) return s;
  if (narrow) {
    shape(128);
    return launch_product<128, A_MN, B_MN, EPI>(ta, tb, p, dev, st);
  }
  return launch_product<256, A_MN, B_MN, EPI>(ta, tb, p, dev, st);
}

template <int EPI>
gtp_status run_update(const Product &p, const Operand &x, const Operand &poly, int64_t count, const Plan &plan,
                      const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (p.tall) return run_product<false, false, EPI>(p, x, poly, count, plan.m, dev, st);
  return run_product<false, true, EPI>(p, poly, x, count, plan.m, dev, st);
}

// The iterations, from X in hi[0] and lo to the last product's epilogue.
template <int EPI>
gtp_status iterate(Product p, const Schedule &s, const Plan &plan, char *ws, int64_t count, int64_t rows, int64_t cols,
                   const gtp::DeviceInfo &dev, cudaStream_t st) {
  const int xs = 12, gs = 12;
  const double top2 = double(s.bound) * s.bound, poly_top = std::fabs(s.b) * top2 + std::fabs(s.c) * top2 * top2;
  const int ps = std::min(14, 15 - int(std::ceil(std::log2(std::max(poly_top, 1.0)))));
  const auto pow2 = [](int e) { return std::ldexp(1.f, e); };
  p.m = int(plan.m), p.tall = rows > cols;
  p.gram = reinterpret_cast<__half *>(ws + plan.gram), p.gram_lo = reinterpret_cast<__half *>(ws + plan.gram_lo);
  p.poly = reinterpret_cast<__half *>(ws + plan.poly);
  p.diag = reinterpret_cast<float *>(ws + plan.diag), p.e = reinterpret_cast<float *>(ws + plan.e);
  p.lo = reinterpret_cast<__half *>(ws + plan.lo);
  p.ldg = plan.ldg, p.planeg = plan.planeg, p.ldx = plan.ldx, p.planex = plan.planex;
  p.gram_scale = pow2(gs), p.gram_inv = pow2(-gs), p.poly_scale = pow2(ps), p.x_scale = pow2(xs), p.x_inv = pow2(-xs);
  p.a = s.a, p.b = s.b, p.c = s.c;
  const Operand gram = {ws + plan.gram, plan.m, plan.m, plan.ldg}, poly = {ws + plan.poly, plan.m, plan.m, plan.ldg};
  for (int k = 0; k < s.steps; ++k) {
    const Operand x = {ws + plan.hi[k & 1], cols, plan.rows, plan.ldx};
    p.symmetric = 1, p.m_dim = p.n_dim = int(plan.m);
    p.alpha = pow2(-2 * xs);
    if (gtp_status e = p.tall ? run_product<true, true, kGram>(p, x, x, count, rows, dev, st)
                              : run_product<false, false, kGram>(p, x, x, count, cols, dev, st))
      return e;
    p.alpha = pow2(-2 * gs);
    if (gtp_status e = run_product<false, false, kPoly>(p, gram, gram, count, plan.m, dev, st)) return e;
    p.symmetric = 0, p.n_fast = p.tall, p.m_dim = int(rows), p.n_dim = int(cols);
    p.alpha = pow2(-ps - xs), p.early = k < 2;
    p.hi = reinterpret_cast<const __half *>(x.base), p.hi_out = reinterpret_cast<__half *>(ws + plan.hi[~k & 1]);
    if (gtp_status e = k + 1 < s.steps ? run_update<kUpdate>(p, x, poly, count, plan, dev, st)
                                       : run_update<EPI>(p, x, poly, count, plan, dev, st))
      return e;
  }
  return GTP_OK;
}

template <typename T, bool VEC, bool STEP>
gtp_status first_of(const Source &s, FirstX f, int64_t count, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const int64_t blocks = (s.items + kPassThreads - 1) / kPassThreads;
  const int64_t fill = std::max<int64_t>(1, int64_t(dev.sm_count) * 8 / count);
  const dim3 squares(unsigned(std::min<int64_t>({(blocks + 3) / 4, fill, kMostParts})), unsigned(count));
  f.parts = int(squares.x);
  if (gtp_status e = gtp::launch_overlapped(squares_kernel<T, VEC, STEP>, squares, kPassThreads, 0, st, "orthogonalize", s, f))
    return e;
  return gtp::launch_overlapped(first_x_kernel<T, VEC, STEP>, dim3(unsigned(std::min(blocks, fill)), unsigned(count)),
                                kPassThreads, 0, st, "orthogonalize", s, f);
}

template <bool STEP>
gtp_status first(Source &s, bool f32, bool vec, const FirstX &f, int64_t count, int64_t rows, int64_t cols,
                 const gtp::DeviceInfo &dev, cudaStream_t st) {
  s.rows = int(rows), s.cols = int(cols);
  s.by_cols = gtp::make_fastdiv(int(vec ? cols / 4 : cols));
  s.items = int(vec ? rows * cols / 4 : rows * cols);
  if (f32) return vec ? first_of<float, true, STEP>(s, f, count, dev, st) : first_of<float, false, STEP>(s, f, count, dev, st);
  return vec ? first_of<__nv_bfloat16, true, STEP>(s, f, count, dev, st)
             : first_of<__nv_bfloat16, false, STEP>(s, f, count, dev, st);
}

bool aligned(const void *p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(to - 1)) == 0; }
int64_t size_of(int dt) { return dt == GTP_F32 ? 4 : 2; }
bool float_type(int dt) { return dt == GTP_F32 || dt == GTP_BF16; }

gtp_status check_sizes(int64_t count, int64_t rows, int64_t cols) {
  if (count < 0 || rows < 0 || cols < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (count > kMostMatrices) return gtp::fail(GTP_E_CAPACITY, "more than %d matrices a call", kMostMatrices);
  if (rows > kMostSide || cols > kMostSide || rows * cols > kMostElements)
    return gtp::fail(GTP_E_SHAPE, "a side above 65536 or a matrix of 2^31 elements");
  return GTP_OK;
}

gtp_status check_workspace(const void *ws, int64_t bytes, const Plan &plan) {
  if (!ws) return gtp::fail(GTP_E_ARG, "null workspace");
  if (!aligned(ws, 256)) return gtp::fail(GTP_E_ALIGN, "workspace must be 256-byte aligned");
  if (bytes < plan.bytes)
    return gtp::fail(GTP_E_CAPACITY, "workspace of %lld bytes, %lld needed", (long long)bytes, (long long)plan.bytes);
  return GTP_OK;
}

FirstX first_x(const Plan &plan, char *ws) {
  FirstX f = {};
  f.part = reinterpret_cast<double *>(ws + plan.part);
  f.hi = reinterpret_cast<__half *>(ws + plan.hi[0]), f.lo = reinterpret_cast<__half *>(ws + plan.lo);
  f.hi_next = reinterpret_cast<__half *>(ws + plan.hi[1]), f.rows = int(plan.rows);
  f.ldx = plan.ldx, f.planex = plan.planex, f.xscale = std::ldexp(1.f, 12);
  return f;
}

}  // namespace

namespace gtp {
gtp_status orthogonalize_wait_word(unsigned int *v, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_ortho_wait_timeouts, sizeof(*v));
  if (e == cudaSuccess && reset) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_ortho_wait_timeouts, &z, sizeof(z));
  }
  if (e != cudaSuccess) return fail(GTP_E_CUDA, "reading the wait-timeout word: %s", cudaGetErrorString(e));
  return GTP_OK;
}
}  // namespace gtp

extern "C" int64_t gtp_orthogonalize_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
  if (check_sizes(count, rows, cols)) return -1;
  if (count == 0 || rows == 0 || cols == 0) return 0;
  return plan_of(count, rows, cols).bytes;
}

extern "C" gtp_status gtp_orthogonalize(const void *src, gtp_dtype src_dt, int64_t src_ld, int64_t src_plane, void *dst,
                                        gtp_dtype dst_dt, int64_t dst_ld, int64_t dst_plane, int64_t count, int64_t rows,
                                        int64_t cols, const float *coefficients, int32_t steps, void *workspace,
                                        int64_t workspace_bytes, gtp_stream stream) {
  gtp::clear_error();
  if (!float_type(src_dt) || !float_type(dst_dt)) return gtp::fail(GTP_E_DTYPE, "dtypes must be F32 or BF16");
  if (gtp_status s = check_sizes(count, rows, cols)) return s;
  Schedule schedule;
  if (gtp_status s = schedule_of(coefficients, steps, &schedule)) return s;
  if (count == 0 || rows == 0 || cols == 0) return GTP_OK;
  if (!src || !dst) return gtp::fail(GTP_E_ARG, "null pointer");
  if (rows == 1) src_ld = dst_ld = cols;
  if (count == 1) src_plane = dst_plane = 0;
  const int64_t most = int64_t(1) << 44;
  if (src_ld < cols || dst_ld < cols || (count > 1 && (src_plane < 0 || dst_plane < (rows - 1) * dst_ld + cols)))
    return gtp::fail(GTP_E_ARG, "a stride below what it steps over");
  if (src_ld > most / rows || dst_ld > most / rows || src_plane > most || dst_plane > most)
    return gtp::fail(GTP_E_SHAPE, "an array spans more than 2^50 elements");
  const int64_t ss = size_of(src_dt), ds = size_of(dst_dt);
  if (!aligned(src, ss) || !aligned(dst, ds)) return gtp::fail(GTP_E_ALIGN, "arrays must be aligned to their elements");
  const Plan plan = plan_of(count, rows, cols);
  if (gtp_status s = check_workspace(workspace, workspace_bytes, plan)) return s;
  const auto span = [&](const void *p, int64_t ld, int64_t plane, int64_t es) {
    return gtp::byte_range(p, ((count - 1) * plane + (rows - 1) * ld + cols) * es);
  };
  const gtp::ByteRange w = gtp::byte_range(workspace, plan.bytes);
  if (gtp::overlap(w, span(src, src_ld, src_plane, ss)) || gtp::overlap(w, span(dst, dst_ld, dst_plane, ds)))
    return gtp::fail(GTP_E_ARG, "the workspace overlaps src or dst");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  cudaStream_t st = gtp::as_stream(stream);
  char *const ws = static_cast<char *>(workspace);
  Source source = {};
  source.src = src, source.ld = src_ld, source.plane = src_plane;
  const bool vec = cols % 4 == 0 && aligned(src, 4 * ss) && src_ld % 4 == 0 && src_plane % 4 == 0;
  if (gtp_status s = first<false>(source, src_dt == GTP_F32, vec, first_x(plan, ws), count, rows, cols, dev, st)) return s;
  Product p = {};
  p.dst = dst, p.ld = dst_ld, p.plane = dst_plane, p.dst_f32 = dst_dt == GTP_F32;
  return iterate<kOut>(p, schedule, plan, ws, count, rows, cols, dev, st);
}

extern "C" gtp_status gtp_muon_step(void *grad_data, gtp_dtype grad_dt, float *momentum, float *master, void *param_data,
                                    int64_t numel, const int64_t *offsets, int64_t count, int64_t rows, int64_t cols,
                                    const gtp_muon_hparams *h, void *workspace, int64_t workspace_bytes, gtp_stream stream) {
  gtp::clear_error();
  if (!float_type(grad_dt)) return gtp::fail(GTP_E_DTYPE, "grad_data must be F32 or BF16");
  if (gtp_status s = check_sizes(count, rows, cols)) return s;
  if (!h) return gtp::fail(GTP_E_ARG, "null hyper-parameters");
  if (!(h->lr >= 0.f) || !(h->weight_decay >= 0.f) || !(h->momentum >= 0.f && h->momentum < 1.f) || !std::isfinite(h->lr) ||
      !std::isfinite(h->weight_decay) || !std::isfinite(h->scale) || !std::isfinite(h->grad_factor))
    return gtp::fail(GTP_E_ARG, "lr, weight_decay >= 0, momentum in [0, 1), scale and grad_factor finite");
  if (h->reserved) return gtp::fail(GTP_E_ARG, "reserved must be 0");
  if ((h->nesterov & ~1) || (h->zero_grad_after & ~1)) return gtp::fail(GTP_E_ARG, "nesterov and zero_grad_after are 0 or 1");
  if (!aligned(h->grad_scale, 4)) return gtp::fail(GTP_E_ALIGN, "grad_scale must be 4-byte aligned");
  Schedule schedule;
  if (gtp_status s = schedule_of(h->coefficients, h->steps, &schedule)) return s;
  if (numel < 0 || numel > (int64_t(1) << 50)) return gtp::fail(GTP_E_ARG, "numel out of range");
  if (count == 0 || rows == 0 || cols == 0) return GTP_OK;
  if (!grad_data || !momentum || !master || !offsets) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t each = rows * cols, gs = size_of(grad_dt);
  bool vec = cols % 4 == 0;
  for (int64_t k = 0; k < count; ++k) {
    if (offsets[k] < 0 || offsets[k] > numel || each > numel - offsets[k])
      return gtp::fail(GTP_E_RANGE, "weight %lld of %lld elements at %lld leaves a buffer of %lld", (long long)k,
                       (long long)each, (long long)offsets[k], (long long)numel);
    for (int64_t j = 0; j < k; ++j)
      if (offsets[j] < offsets[k] + each && offsets[k] < offsets[j] + each)
        return gtp::fail(GTP_E_RANGE, "weights %lld and %lld overlap", (long long)j, (long long)k);
    vec = vec && offsets[k] % 4 == 0;
  }
  if (!aligned(grad_data, gs) || !aligned(momentum, 4) || !aligned(master, 4) || !aligned(param_data, 2))
    return gtp::fail(GTP_E_ALIGN, "arrays must be aligned to their elements");
  const Plan plan = plan_of(count, rows, cols);
  if (gtp_status s = check_workspace(workspace, workspace_bytes, plan)) return s;
  const gtp::ByteRange r[5] = {gtp::byte_range(grad_data, numel * gs), gtp::byte_range(momentum, 4 * numel),
                               gtp::byte_range(master, 4 * numel), gtp::byte_range(workspace, plan.bytes),
                               gtp::byte_range(param_data, param_data ? 2 * numel : 0)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (gtp::overlap(r[i], r[j])) return gtp::fail(GTP_E_ARG, "two of the arrays overlap");
    if (h->grad_scale && gtp::overlap(r[i], gtp::byte_range(h->grad_scale, 4)))
      return gtp::fail(GTP_E_ARG, "grad_scale lies in one of the arrays");
  }
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  cudaStream_t st = gtp::as_stream(stream);
  char *const ws = static_cast<char *>(workspace);
  Source source = {};
  source.grad = grad_data, source.momentum = momentum, source.grad_scale = h->grad_scale;
  source.mu = h->momentum, source.factor = h->grad_factor, source.nesterov = h->nesterov, source.zero_grad = h->zero_grad_after;
  Product p = {};
  p.master = master, p.param = static_cast<__nv_bfloat16 *>(param_data);
  p.keep = float(1.0 - double(h->lr) * double(h->weight_decay)), p.rate = float(double(h->lr) * double(h->scale));
  for (int64_t k = 0; k < count; ++k) source.offset[k] = p.offset[k] = offsets[k];
  vec = vec && aligned(grad_data, 4 * gs) && aligned(momentum, 16);
  if (gtp_status s = first<true>(source, grad_dt == GTP_F32, vec, first_x(plan, ws), count, rows, cols, dev, st)) return s;
  return iterate<kStep>(p, schedule, plan, ws, count, rows, cols, dev, st);
}
