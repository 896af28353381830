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
// Three products an iteration.  A and A^2 are symmetric: only tiles on and above the diagonal are computed, and written
// twice.
//
// Precision.  The operands are fp16, whose 11 bits err an eighth of bf16's at the same rate; all values here are bounded
// (|X|_2 stays near 1), so powers of two hold them in fp16's range.  Three choices keep rounding away from where the
// polynomial's terms cancel (a + b + c = 0.7 out of terms up to 4.8):
//   - the diagonals of A and B never become fp16: d = diag(A) and e = a + diag(B) stay fp32 vectors, with A = d + A'
//     the square is d^2 + (d_i + d_j) A' + A'^2, and X <- e X + B' X;
//   - the X of the linear term is fp16 high part + fp16 low part (22 bits); the products read the high part alone.  The
//     low part is scaled by e where X is nearly orthogonal (B' is small there: what its product leaves out is small),
//     but by a alone in the first iterations, where small singular values, on which e acts as far less than a + B does,
//     still grow a-fold each.  Those that matter in the end are small until the last three (`early_of`);
//   - A' enters B' with a low part of its own (the square reads the high part).
// Against fp64, relative error of the result at five steps: 1e-4 to 1.5e-3 over Gaussian, row-scaled and low-rank matrices with
// sides of 16 and more (rank 8 and 1e-3 of noise in 16 x 4096 2.6e-3; with a side of 2 to 9e-3); without the first two
// choices 2e-3 to 9e-3, with bf16 operands 1.4e-2 to 6e-2.  A bf16 result's own rounding is 1.7e-3.  Later iterations carry
// the roundings of earlier ones on by the polynomial's slopes: mostly 3e-3 at ten steps and 4e-3 at sixteen.
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
#include "smem_base.h"
#include "tensor_map.h"

namespace gtp {
void clear_error();
}

namespace {

using namespace gtp::ptx;

__device__ unsigned int g_ortho_wait_timeouts;  // this unit's part of gtp_wait_timeouts' word

constexpr int kMostMatrices = 64, kMostSteps = 16;
constexpr int kCounters = 3 * kMostSteps * kMostMatrices;  // of a launch: one a product and matrix

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
  unsigned int *arrived;  // the products' counters, cleared here
};

// Elements as they lie in memory, until they are wanted: a load whose value is converted at once is waited for at once.
template <typename T, bool VEC>
struct Raw {
  T v;
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = float(v); }
};
template <>
struct Raw<float, true> {
  float4 v;
  __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
};
template <>
struct Raw<__nv_bfloat16, true> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
};

// Item i of matrix k, four consecutive elements of a row with VEC, else one: the matrix's own, or the gradient and the
// momentum that the step's u comes from.
template <typename T, bool VEC, bool STEP>
struct Item {
  static constexpr int E = VEC ? 4 : 1;
  Raw<T, VEC> raw;
  Raw<float, VEC> old;  // the momentum, of a step
  float g[E], m[E];
  int row, col;

  __device__ __forceinline__ int64_t at(const Source &s, int k) const { return s.offset[k] + int64_t(row) * s.cols + col; }
  __device__ __forceinline__ void load(const Source &s, int k, int i) {
    row = gtp::fast_div(i, s.by_cols);
    col = (i - row * (s.cols / E)) * E;
    raw.load(STEP ? static_cast<const T *>(s.grad) + at(s, k) : static_cast<const T *>(s.src) + k * s.plane + row * s.ld + col);
    if constexpr (STEP) old.load(s.momentum + at(s, k));
  }
  // The values to orthogonalise, in g.  FIRST: the pass that writes the momentum; the second one finds it written and
  // clears the gradient.
  template <bool FIRST>
  __device__ __forceinline__ void finish(const Source &s, int k, float g_scale) {
    raw.get(g);
    if constexpr (STEP) {
      old.get(m);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        g[e] *= g_scale;
        if (FIRST) m[e] = fmaf(s.mu, m[e], (1.f - s.mu) * g[e]);
        g[e] = s.nesterov ? fmaf(s.mu, m[e], (1.f - s.mu) * g[e]) : m[e];
      }
      if (FIRST) {
        float *const mp = s.momentum + at(s, k);
        if constexpr (VEC) *reinterpret_cast<float4 *>(mp) = make_float4(m[0], m[1], m[2], m[3]);
        else *mp = m[0];
      } else if (s.zero_grad) {
        T *const gp = static_cast<T *>(s.grad) + at(s, k);
        if constexpr (!VEC) gp[0] = T(0.f);
        else if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(gp) = make_float4(0.f, 0.f, 0.f, 0.f);
        else *reinterpret_cast<uint2 *>(gp) = make_uint2(0u, 0u);
      }
    }
  }
};

// The sum over the block, in thread 0 (fp64 is slow here: nothing of it in more threads than have to).
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double sums[32];
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  if (threadIdx.x == 0)
    for (int w = 0; w < int(blockDim.x >> 5); ++w) v += sums[w];
  return v;
}

constexpr int kPassThreads = 256, kFlight = 4;  // items of a thread whose loads are under way together

// Sums of squares, a block's part each (and the new momentum).
template <typename T, bool VEC, bool STEP>
__global__ void __launch_bounds__(kPassThreads)
    squares_kernel(const __grid_constant__ Source s, const __grid_constant__ FirstX f) {
  allow_dependents();
  wait_prior_grid();
  const float g_scale = STEP ? s.factor * (s.grad_scale ? *s.grad_scale : 1.f) : 1.f;
  double total = 0;
  const int64_t step = int64_t(gridDim.x) * kPassThreads;
  for (int64_t i0 = int64_t(blockIdx.x) * kPassThreads + threadIdx.x; i0 < s.items; i0 += kFlight * step) {
    Item<T, VEC, STEP> x[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      if (i0 + j * step < s.items) x[j].load(s, blockIdx.y, int(i0 + j * step));
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      if (i0 + j * step < s.items) {
        x[j].template finish<true>(s, blockIdx.y, g_scale);
#pragma unroll
        for (int e = 0; e < Item<T, VEC, STEP>::E; ++e) sum = fmaf(x[j].g[e], x[j].g[e], sum);
      }
    }
    if (sum >= 0x1p-100f && sum <= 0x1p120f) {
      total += double(sum);
    } else {  // squares that fp32 does not hold, or not in full: of elements below 2^-50 and above 2^57 times a power of two
      const float by = sum < 1.f ? 0x1p100f : 0x1p-72f;
      const double back = sum < 1.f ? 0x1p-200 : 0x1p144;
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < kFlight; ++j)
        if (i0 + j * step < s.items) {
#pragma unroll
          for (int e = 0; e < Item<T, VEC, STEP>::E; ++e) sum = fmaf(x[j].g[e] * by, x[j].g[e] * by, sum);
        }
      total = fma(double(sum), back, total);
    }
  }
  total = block_sum(total);
  if (threadIdx.x == 0) f.part[blockIdx.y * gridDim.x + blockIdx.x] = total;
}

// X = G / |G|_F as fp16 high and low parts, times a power of two.  A matrix of zeros stays zero; one with NaN or Inf
// becomes NaN.
template <typename T, bool VEC, bool STEP>
__global__ void __launch_bounds__(kPassThreads)
    first_x_kernel(const __grid_constant__ Source s, const __grid_constant__ FirstX f) {
  allow_dependents();
  wait_prior_grid();
  const float g_scale = STEP ? s.factor * (s.grad_scale ? *s.grad_scale : 1.f) : 1.f;
  double total = 0;
  for (int p = threadIdx.x; p < f.parts; p += kPassThreads) total += f.part[blockIdx.y * f.parts + p];
  total = block_sum(total);
  __shared__ float scale[2];  // 1 / |G|: a power of two that its elements take first, exactly, and what fp32 then holds
  if (threadIdx.x == 0) {
    const double inv = total == 0 ? 0. : isfinite(total) ? double(f.xscale) / sqrt(total) : double(nanf(""));
    const bool large = inv > 0x1p100, small = inv < 0x1p-100;
    scale[0] = large ? 0x1p100f : small ? 0x1p-64f : 1.f;
    scale[1] = float(inv * (large ? 0x1p-100 : small ? 0x1p64 : 1.));
  }
  __syncthreads();
  const float p = scale[0], r = scale[1];
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < kCounters; i += kPassThreads) f.arrived[i] = 0;
  const int step = int(gridDim.x) * kPassThreads, me = int(blockIdx.x) * kPassThreads + int(threadIdx.x);
  const int64_t zeros = (f.rows - s.rows) * f.ldx / 8;  // in both buffers that take turns as the products' X
  for (int64_t i = me; i < zeros; i += step) {
    const int64_t at = blockIdx.y * f.planex + s.rows * f.ldx + 8 * i;
    *reinterpret_cast<uint4 *>(f.hi + at) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4 *>(f.hi_next + at) = make_uint4(0, 0, 0, 0);
  }
  for (int64_t i0 = me; i0 < s.items; i0 += int64_t(kFlight) * step) {
    Item<T, VEC, STEP> x[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      if (i0 + int64_t(j) * step < s.items) x[j].load(s, blockIdx.y, int(i0 + int64_t(j) * step));
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      if (i0 + int64_t(j) * step >= s.items) continue;
      x[j].template finish<false>(s, blockIdx.y, g_scale);
      const int64_t at = blockIdx.y * f.planex + x[j].row * f.ldx + x[j].col;
      constexpr int E = Item<T, VEC, STEP>::E;
      __half hi[E], lo[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = x[j].g[e] * p * r;
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
}

// --------------------------------------------------------------------------- the products

// All products of a call in one cooperative launch of CTA pairs.  A phase is one product of one iteration over all
// matrices; its pair tiles go round the pairs, on from where the phase before ended.  A matrix's product waits for that
// matrix's product before alone: every CTA counts off each tile it has finished (arrived[phase][matrix], cleared by
// first_x_kernel), so that with several matrices the pairs go from phase to phase without a pause.  No wait can close
// a circle: a pair takes its tiles in the order of phases, and waits only for earlier phases.
//
// Inside a CTA: warp 0 and warp 2 copy A and B tiles to a ring of shared-memory stages, warp 1 of the even CTA issues the
// M = 256 MMAs of the pair into one of two accumulators, warp 3 waits for phases, warps 4-11 finish the tiles: 32 x 32
// chunks of the accumulator meet the old values (A', or X's two parts) that a tensor copy brought to the warp's own
// staging slot one chunk ahead, and the new ones leave through the same slot.
constexpr int BK = 64, UK = 16, BMC = 128, BMP = 256, BN = 256;
constexpr int BOX = 64 * 64 * 2;  // one tensor copy: 64 rows of 128 bytes, either majorness
constexpr int A_STAGE = BMC * BK * 2, STAGE = 2 * A_STAGE, STAGES = 5;
constexpr int kEpilogueWarps = 8, kThreads = 128 + 32 * kEpilogueWarps;
constexpr int PART = 32 * 32 * 2, SLOT = 2 * PART, SLOTS = 2;  // a chunk of fp16; high and low part of one; a warp's
constexpr int SMEM_OPS = STAGES * STAGE, SMEM_SLOTS = kEpilogueWarps * SLOTS * SLOT;
constexpr int SMEM_VEC = kEpilogueWarps * 32 * 4, SMEM_CTRL = 512;
constexpr int SMEM_TOTAL = SMEM_OPS + SMEM_SLOTS + SMEM_VEC + SMEM_CTRL;
static_assert(SMEM_TOTAL <= 232448, "shared memory per block");

enum Kind { kGram, kPoly, kUpdate };

struct Phase {
  int units, full;       // tiles, the last ones (from `full` on) as two half-wide units each
  int each, tiles_m, tiles_n, k_blocks;
  int a_rows, b_rows;    // a matrix's rows in either operand
  int m_dim, n_dim, out_rows;  // of the output; its rows in memory
};

struct Maps {
  CUtensorMap x[2], gram, poly;                                   // operands: boxes of 64 rows of 64 elements
  CUtensorMap x_tall[2], gram_tall, poly_tall;                    // and of 128 rows
  CUtensorMap c_hi[2], c_lo, c_gram, c_gram_lo, c_poly;           // 32 x 32 chunks
};
static_assert(sizeof(Maps) == 14 * sizeof(CUtensorMap), "prefetched one by one");

struct Args {
  Phase phase[3];
  int count, steps, m, step;  // step: the last product moves the master instead of writing dst
  int early;             // the iterations that scale X's low part by a
  unsigned int *arrived;
  float *diag, *e;       // [count][m]
  // powers of two: what makes the accumulators, A', B' and X true values and the reverse
  float x_scale, x_inv, gram_scale, gram_inv, poly_scale, poly_inv;
  float a, b, c;
  void *dst;
  int64_t ld, plane;
  int dst_f32;
  float *master;
  __nv_bfloat16 *param;
  float keep, rate;      // 1 - lr wd, lr scale
  int64_t offset[kMostMatrices];
};

// A unit's matrix, its first row of 256 and first column, and whether it is half as wide; false where it lies beside the
// output (the second half of a narrow last tile).
template <bool SYMMETRIC, bool N_FAST>
__device__ __forceinline__ bool decode(const Phase &p, int u, int &k, int &row, int &col, bool &half) {
  int t = u;
  int h = 0;
  half = u >= p.full;
  if (half) {
    t = p.full + ((u - p.full) >> 1);
    h = (u - p.full) & 1;
  }
  k = t / p.each;
  t -= k * p.each;
  int tm, tn;
  if (SYMMETRIC) {  // row tm of the tiles on and above the diagonal has tiles_n - tm of them
    tm = 0;
    while (t >= p.tiles_n - tm) t -= p.tiles_n - tm++;
    tn = tm + t;
  } else if (N_FAST) {
    tm = t / p.tiles_n;
    tn = t - tm * p.tiles_n;
  } else {
    tn = t / p.tiles_m;
    tm = t - tn * p.tiles_m;
  }
  row = tm * BMP;
  col = tn * BN + h * (BN / 2);
  return col < p.n_dim;
}

template <bool TALL>
__device__ __forceinline__ bool decode(const Phase &p, int kind, int u, int &k, int &row, int &col, bool &half) {
  return kind == kUpdate ? decode<false, TALL>(p, u, k, row, col, half) : decode<true, false>(p, u, k, row, col, half);
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

__device__ __forceinline__ unsigned int load_acquire(const unsigned int *p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(unsigned int *p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {  // without a pause
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all_but_one() { asm volatile("cp.async.bulk.wait_group 1;" ::: "memory"); }

// The pair's first unit of the phase that follows one of `units`.
__device__ __forceinline__ int next_first(int first, int units, int step) {
  first -= units % step;
  return first < 0 ? first + step : first;
}

// Waits until warp 3 has said that this CTA may start `phase` (of newton_schulz_kernel: phase * count + matrix); false
// when the CTA gives up.
__device__ __forceinline__ bool wait_ready(volatile int *ready, int phase, volatile int *abort_flag, unsigned int *err) {
  if (*ready < phase) {
    const uint64_t t0 = globaltimer_ns();
    uint32_t spins = 0;
    while (*ready < phase) {
      if ((++spins & 63u) == 0) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicOr(err, 0x10u);
          return false;
        }
      }
    }
  }
  __threadfence_block();
  return true;
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t bits2(float2 v) { return uint64_t(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x); }
__device__ __forceinline__ float2 float2_of(uint64_t v) { return make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32))); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// The low part of a pair whose high part is `high`: what fp16 left over.
__device__ __forceinline__ uint32_t low2(float2 v, uint32_t high) {
  const float2 h = unpack2(high), l = add2(v, make_float2(-h.x, -h.y));
  return pack2(l.x, l.y);
}
__device__ __forceinline__ float2 pair_of(const uint32_t (&r)[16], int i) { return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])); }

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// A 32 x 32 chunk of fp16 lies as the copies' 64-byte swizzle has it: the 16-byte piece j (eight columns) of row r at
// r * 64 + 16 (j ^ (r / 2 % 4)).
__device__ __forceinline__ int piece_at(int row, int j) { return row * 64 + ((j ^ ((row >> 1) & 3)) << 4); }

// The chunk in `from` transposed into `to`: this lane's row becomes column `lane`.
__device__ __forceinline__ void transpose_chunk(const uint8_t *from, uint8_t *to, int lane) {
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const uint4 v = *reinterpret_cast<const uint4 *>(from + piece_at(lane, j));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint16_t *>(to + piece_at(8 * j + i, lane >> 3) + 2 * (lane & 7)) =
          uint16_t(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
  }
}

// The last product's values of a chunk, true values in fp32 at `staged` (row r's 16-byte piece j at r * 128 + 16 (j ^ r
// % 8)), out in whole row segments: eight lanes a row of 32, four values a lane.
__device__ __forceinline__ void write_out(const Args &a, int m_dim, int n_dim, const uint8_t *staged, int lane, int k,
                                          int row0, int col) {
  const int j = lane & 7, c = col + 4 * j;
  const int n = min(4, n_dim - c);
  if (n <= 0) return;
  const int64_t ld = a.step ? n_dim : a.ld;
  const int64_t base = (a.step ? a.offset[k] : k * a.plane) + (row0 + (lane >> 3)) * ld + c;
  const bool in4 = n == 4 && ld % 4 == 0;
#pragma unroll 1
  for (int i0 = 0; i0 < 8; i0 += 4) {
    float4 m[4];
    if (a.step) {
      const bool wide = in4 && (reinterpret_cast<uintptr_t>(a.master + base) & 15) == 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float *const o = a.master + base + 4 * (i0 + i) * ld;
        if (row0 + 4 * (i0 + i) + (lane >> 3) >= m_dim) continue;
        if (wide) m[i] = *reinterpret_cast<const float4 *>(o);
        else m[i] = make_float4(o[0], n > 1 ? o[1] : 0.f, n > 2 ? o[2] : 0.f, n > 3 ? o[3] : 0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * (i0 + i) + (lane >> 3);
      if (row0 + r >= m_dim) continue;
      const int64_t at = base + 4 * (i0 + i) * ld;
      float4 v = *reinterpret_cast<const float4 *>(staged + r * 128 + ((j ^ (r & 7)) << 4));
      if (a.step)
        v = make_float4(fmaf(a.keep, m[i].x, -a.rate * v.x), fmaf(a.keep, m[i].y, -a.rate * v.y),
                        fmaf(a.keep, m[i].z, -a.rate * v.z), fmaf(a.keep, m[i].w, -a.rate * v.w));
      const float y[4] = {v.x, v.y, v.z, v.w};
      float *const o = a.step ? a.master + at : a.dst_f32 ? static_cast<float *>(a.dst) + at : nullptr;
      if (o) {
        if (in4 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
          *reinterpret_cast<float4 *>(o) = v;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < n) o[q] = y[q];
        }
      }
      __nv_bfloat16 *const b = a.step ? (a.param ? a.param + at : nullptr)
                                      : a.dst_f32 ? nullptr : static_cast<__nv_bfloat16 *>(a.dst) + at;
      if (b) {
        if (in4 && (reinterpret_cast<uintptr_t>(b) & 7) == 0) {
          const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
          *reinterpret_cast<uint2 *>(b) = *reinterpret_cast<const uint2 *>(w);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < n) b[q] = __float2bfloat16_rn(y[q]);
        }
      }
    }
  }
}

// EDGE: element `diagonal` of the sixteen is on the diagonal, which is kept apart (true value) and left out, and so are
// elements from `limit` on.
template <bool EDGE>
__device__ __forceinline__ void leave_out(const uint32_t (&r)[16], float alpha, int diagonal, int limit, float &at_diagonal,
                                      float2 (&x)[8]) {
  if constexpr (EDGE) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i == diagonal) at_diagonal = __uint_as_float(r[i]) * alpha;
      if (i == diagonal || i >= limit) (i & 1 ? x[i >> 1].y : x[i >> 1].x) = 0.f;
    }
  }
}
// Sixteen elements of a row of A' out of its accumulator, times `scale`.
template <bool EDGE>
__device__ __forceinline__ void gram_row(const uint32_t (&r)[16], float scale, float alpha, int diagonal, int limit,
                                         float &at_diagonal, float2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = mul2(pair_of(r, 2 * i), both(scale));
  leave_out<EDGE>(r, alpha, diagonal, limit, at_diagonal, x);
}

// The same of B' = b A' + c ((d_i + d_j) A' + A'^2): g holds A' and r its square, in their own scales;
// k = {b + c d_i, c, c}, each with the powers of two that make the sum B' in its scale.
template <bool EDGE>
__device__ __forceinline__ void poly_row(const uint32_t (&r)[16], const float2 (&g)[8], const float2 (&dj)[8], const float (&k)[3],
                                         float alpha, int diagonal, int limit, float &at_diagonal, float2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = fma2(g[i], fma2(both(k[1]), dj[i], both(k[0])), mul2(pair_of(r, 2 * i), both(k[2])));
  leave_out<EDGE>(r, alpha, diagonal, limit, at_diagonal, x);
}

__device__ __forceinline__ void load16(const float *p, float2 (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 f = *reinterpret_cast<const float4 *>(p + 4 * q);
    x[2 * q] = make_float2(f.x, f.y), x[2 * q + 1] = make_float2(f.z, f.w);
  }
}

// A chunk of the update, from the accumulator at `taddr` and the old X in hi and lo: the new X in their place, or (last)
// true values in `staged`.  v: e of the chunk's columns (TALL), own: e of this lane's row; inside: that row exists (those
// that fill a contraction's last block keep the zeros that came).  Sixteen columns at a time: the code of a phase stays
// small.
template <bool TALL>
__device__ __forceinline__ void update_chunk(const Args &a, uint32_t taddr, uint8_t *hi, uint8_t *lo, uint8_t *staged,
                                             const float *v, float own, bool inside, bool early, bool last, int lane) {
  const float alpha = a.poly_inv;  // the accumulator in X's scale
#pragma unroll 1
  for (int j = 0; j < 4; j += 2) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(taddr + uint32_t(8 * j), r);
    uint32_t h[8], l[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 hv = *reinterpret_cast<const uint4 *>(hi + piece_at(lane, j + q));
      const uint4 lv = *reinterpret_cast<const uint4 *>(lo + piece_at(lane, j + q));
      h[4 * q] = hv.x, h[4 * q + 1] = hv.y, h[4 * q + 2] = hv.z, h[4 * q + 3] = hv.w;
      l[4 * q] = lv.x, l[4 * q + 1] = lv.y, l[4 * q + 2] = lv.z, l[4 * q + 3] = lv.w;
    }
    float2 e[8], x[8];
    if (TALL) {
      load16(v + 8 * j, e);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = both(own);
    }
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = mul2(pair_of(r, 2 * i), both(alpha));
    if (early) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fma2(e[i], unpack2(h[i]), fma2(both(a.a), unpack2(l[i]), x[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fma2(e[i], add2(unpack2(h[i]), unpack2(l[i])), x[i]);
    }
    if (last) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(staged + lane * 128 + (((2 * j + i) ^ (lane & 7)) << 4)) =
            make_float4(x[2 * i].x * a.x_inv, x[2 * i].y * a.x_inv, x[2 * i + 1].x * a.x_inv, x[2 * i + 1].y * a.x_inv);
      continue;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = pack2(x[i].x, x[i].y);
      l[i] = low2(x[i], h[i]);
    }
    if (inside) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        *reinterpret_cast<uint4 *>(hi + piece_at(lane, j + q)) = make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
        *reinterpret_cast<uint4 *>(lo + piece_at(lane, j + q)) = make_uint4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]);
      }
    }
  }
}

// The same chunk on its way: a copy of both parts to X's next buffers, or the result written out.  The whole warp.
__device__ __forceinline__ void send_chunk(const Args &a, const CUtensorMap *to_hi, const CUtensorMap *to_lo, uint8_t *hi,
                                           uint8_t *lo, const uint8_t *staged, bool last, int lane, int k, int m_dim, int n_dim,
                                           int stand, int row0, int col) {
  if (!last) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(to_hi, hi, col, k * stand + row0);
      tma_store_2d(to_lo, lo, col, k * stand + row0);
      bulk_commit_group();
    }
  } else {
    __syncwarp();
    write_out(a, m_dim, n_dim, staged, lane, k, row0, col);
    fence_proxy_async_smem();  // before a copy lands where this was
    __syncwarp();
  }
}

template <bool TALL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    newton_schulz_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem_at_1024[];  // the host checks that it starts there
  uint8_t *sA = smem_at_1024, *sB = sA + STAGES * A_STAGE, *slots = sA + SMEM_OPS;
  float(*const vec)[32] = reinterpret_cast<float(*)[32]>(slots + SMEM_SLOTS);  // d or e of a chunk's columns, a warp each
  uint64_t *full = reinterpret_cast<uint64_t *>(vec + kEpilogueWarps);
  uint64_t *empty = full + STAGES;
  uint64_t *tfull = empty + STAGES;
  uint64_t *tempty = tfull + 2;
  uint64_t *drained = tempty + 2;
  uint64_t *cfull = drained + 1;  // [warp][slot]: a chunk's old values have landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(cfull + SLOTS * kEpilogueWarps);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *ready = abort_flag + 1;
  int *finished = const_cast<int *>(ready + 1);  // [4], by units in turn: the warps that have finished their part of one
  static_assert((2 * STAGES + 5 + SLOTS * kEpilogueWarps) * 8 + 28 <= SMEM_CTRL, "control block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = int(blockIdx.x >> 1), step = int(gridDim.x >> 1), phases = 3 * a.steps;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpilogueWarps);
    }
    mbar_init(drained, 1);
    for (int i = 0; i < SLOTS * kEpilogueWarps; ++i) mbar_init(&cfull[i], 1);
    *abort_flag = 0;
    *ready = 0;
    for (int i = 0; i < 4; ++i) finished[i] = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane < 14) tma_prefetch_desc(reinterpret_cast<const CUtensorMap *>(&maps) + lane);
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

  if (warp == 0 || warp == 2) {
    if (lane == 0) {  // ------------------------------------ producers (both CTAs): warp 0 A, warp 2 B
      // One copy a block and thread, two where rows run along the contraction, and little else: the threads' issuing bounds
      // the kernel where there is more (two boxes of 64 rows in place of one of 128, and the arming kept in an array: 590
      // cycles a block for the 256 of a half-wide unit's MMAs, now 440).
      const bool is_a = warp == 0;
      int stage = 0;
      uint32_t parity = 0, armed = 0, armed_parity = 0;  // bit s: stage s has been armed, and for which phase
      const uint32_t bars = mapa_shared(full, 0);
      bool ok = true;
      for (int ph = 0, kind = 0, first = pair; ok && ph < phases;
           ++ph, first = next_first(first, a.phase[kind].units, step), kind = kind == 2 ? 0 : kind + 1) {
        const Phase &p = a.phase[kind];
        if (first >= p.units) continue;
        const int xi = (ph / 3) & 1;
        const bool mn = kind == kGram ? TALL : kind == kUpdate && !is_a && !TALL;  // rows of the box run along K
        const bool of_x = kind == kGram || (kind == kUpdate && is_a == TALL);
        const CUtensorMap *map = of_x ? &maps.x[xi] : kind == kPoly ? &maps.gram : &maps.poly;
        const CUtensorMap *tall_map = of_x ? &maps.x_tall[xi] : kind == kPoly ? &maps.gram_tall : &maps.poly_tall;
        const int rows = is_a ? p.a_rows : p.b_rows;
        for (int u = first; ok && u < p.units; u += step) {
          int k, row, col;
          bool half;
          if (!decode<TALL>(p, kind, u, k, row, col, half)) continue;
          // this CTA's 128 rows of A, 128 or 64 of B
          const bool whole = is_a || !half;
          const int i0 = is_a ? row + BMC * int(rank) : col + (half ? 64 : 128) * int(rank), r0 = k * rows;
          const uint32_t bytes = half ? 2u * (A_STAGE + BOX) : 2u * STAGE;
          const CUtensorMap *const use = whole && !mn ? tall_map : map;
          if (ph > 0 && !(ok = wait_ready(ready, ph * a.count + k, abort_flag, err))) break;
          int cx = mn ? i0 : 0, cy = mn ? r0 : r0 + i0;
          const int dx = mn ? 0 : BK, dy = mn ? BK : 0;
          uint8_t *const base = is_a ? sA : sB;
          for (int kb = 0; kb < p.k_blocks; ++kb) {
            if (!mbar_wait(&empty[stage], parity ^ 1u, abort_flag, err, 0x1u)) {
              ok = false;
              break;
            }
            if (is_a && rank == 0) {  // the even CTA's barrier counts both CTAs' bytes
              mbar_arrive_expect_tx_relaxed(&full[stage], bytes);
              armed |= 1u << stage;
              armed_parity = (armed_parity & ~(1u << stage)) | parity << stage;
            }
            uint8_t *const to = base + stage * A_STAGE;
            tma_load_2d_pair(use, bars + 8 * stage, to, cx, cy);
            if (mn && whole) tma_load_2d_pair(use, bars + 8 * stage, to + BOX, cx + 64, cy);
            cx += dx, cy += dy;
            if (++stage == STAGES) {
              stage = 0;
              parity ^= 1u;
            }
          }
        }
      }
      for (int s = 0; s < STAGES; ++s)  // every armed copy has landed before the pair leaves
        if (armed >> s & 1) drain(&full[s], armed_parity >> s & 1);
    }
  } else if (warp == 1) {  // ---------------------------------------------- MMA (the even CTA)
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t parity = 0, acc_parity = 0;
      bool ok = true;
      for (int ph = 0, kind = 0, first = pair; ok && ph < phases;
           ++ph, first = next_first(first, a.phase[kind].units, step), kind = kind == 2 ? 0 : kind + 1) {
        const Phase &p = a.phase[kind];
        const bool a_mn = kind == kGram && TALL, b_mn = a_mn || (kind == kUpdate && !TALL);
        for (int u = first; ok && u < p.units; u += step) {
          int k, row, col;
          bool half;
          if (!decode<TALL>(p, kind, u, k, row, col, half)) continue;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_parity ^ 1u, abort_flag, err, 0x2u))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + uint32_t(acc * BN);
          const uint32_t idesc = idesc_f16_f32(BMP, half ? BN / 2 : BN, a_mn, b_mn);
          // from one K = 16 slice of a stage to the next: 16 rows of 128 bytes, or 32 bytes of each row
          const uint32_t da = a_mn ? UK * 128 : UK * 2, db = b_mn ? UK * 128 : UK * 2;
          for (int kb = 0; kb < p.k_blocks; ++kb) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], parity, abort_flag, err, 0x4u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one_sync()) {
              const uint32_t a0 = smem_u32(sA + stage * A_STAGE), b0 = smem_u32(sB + stage * A_STAGE);
#pragma unroll
              for (int i = 0; i < BK / UK; ++i) {
                const uint64_t ad = sdesc_sw128(a0 + i * da, a_mn ? BOX : 16, 1024);
                const uint64_t bd = sdesc_sw128(b0 + i * db, b_mn ? BOX : 16, 1024);
                mma_f16_pair(d, ad, bd, idesc, (kb > 0 || i > 0) ? 1u : 0u);
              }
              mma_commit_pair(&empty[stage], 0x3);
            }
            __syncwarp();
            if (++stage == STAGES) {
              stage = 0;
              parity ^= 1u;
            }
          }
          if (!ok) break;
          if (elect_one_sync()) mma_commit_pair(&tfull[acc], 0x3);
          __syncwarp();
          if (++acc == 2) {
            acc = 0;
            acc_parity ^= 1u;
          }
        }
      }
      if (elect_one_sync()) mma_commit_pair(drained, 0x3);  // both CTAs learn when every MMA has finished
      __syncwarp();
    }
    if (lane == 0) drain(drained, 0);
  } else if (warp == 3) {
    if (lane == 0) {  // ---------------------------------------------------- the phases' order
      bool ok = true;
      for (int ph = 0, kind = 0, first = pair; ok && ph < phases;
           ++ph, first = next_first(first, a.phase[kind].units, step), kind = kind == 2 ? 0 : kind + 1) {
        if (ph == 0) continue;
        const Phase &p = a.phase[kind], &before = a.phase[kind == 0 ? 2 : kind - 1];
        int said = -1;
        for (int u = first; ok && u < p.units; u += step) {
          int k, row, col;
          bool half;
          if (!decode<TALL>(p, kind, u, k, row, col, half) || k == said) continue;
          // units of the matrix in the phase before, counted off by both CTAs
          const int whole = min(max(before.full - k * before.each, 0), before.each);
          const unsigned int all = 2u * unsigned(2 * before.each - whole);
          const uint64_t t0 = globaltimer_ns();
          while (load_acquire(&a.arrived[(ph - 1) * a.count + k]) < all) {
            if (*abort_flag) ok = false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
              atomicOr(err, 0x200u);
              ok = false;
            }
            if (!ok) break;
          }
          if (!ok) {
            *abort_flag = 1;
            break;
          }
          // what the other CTAs' copies wrote, before this CTA's copies read it
          fence_proxy_async_global();
          __threadfence_block();
          *ready = ph * a.count + k;
          said = k;
        }
      }
    }
  } else {  // -------------------------------------------------------------- finishing the tiles (both CTAs)
    const int ew = warp - 4, quarter = warp & 3, side = ew >> 2;
    uint8_t *const mine = slots + ew * SLOTS * SLOT;
    uint64_t *const cbar = cfull + SLOTS * ew;
    float *const v = vec[ew];
    int acc = 0, slot = 0;
    int ahead = 0;                         // chunks fetched and not yet worked on, from `slot` on
    uint32_t acc_parity = 0, cparity = 0;  // bit s: the parity that slot s's next copy completes
    int flying = 0;                        // bit s: a copy into slot s that nobody has waited for
    bool ok = true;
    // The counter of a unit whose chunks have left and may not have arrived: this warp is done with it when they have, d
    // and e having been written by its lanes before the warp's barrier.  The last of the warps counts the unit off and
    // releases what it and, through `finished`, the others have written.  No warp gets to a unit four further on before
    // all have: a unit's accumulator is the one of two before.
    unsigned int *owed = nullptr;
    int done = 0;
    const auto settle = [&](bool all) {  // else all but the chunk sent last, which is another unit's
      if (!owed) return;
      if (lane == 0) {
        if (all) bulk_wait_all();
        else bulk_wait_all_but_one();
      }
      __syncwarp();
      if (lane == 0) {
        __threadfence_block();
        if ((atomicAdd(&finished[done & 3], 1) & (kEpilogueWarps - 1)) == kEpilogueWarps - 1) {
          __threadfence_block();
          add_release(owed);
        }
      }
      ++done;
      owed = nullptr;
    };
    for (int ph = 0, kind = 0, first = pair; ok && ph < phases;
           ++ph, first = next_first(first, a.phase[kind].units, step), kind = kind == 2 ? 0 : kind + 1) {
      const Phase &p = a.phase[kind];
      if (first >= p.units) continue;
      const bool last = ph + 1 == phases, early = ph < 3 * a.early;
      unsigned int *const counters = a.arrived + ph * a.count;
      const CUtensorMap *const from_hi = kind == kPoly ? &maps.c_gram : &maps.c_hi[(ph / 3) & 1];
      const CUtensorMap *const from_lo = kind == kPoly ? &maps.c_gram_lo : &maps.c_lo;
      // Old values are fetched in the order in which chunks are worked on: the next chunk's before this one's new values
      // leave (in the last product after it, which lends the other slot to the result).
      const auto exists = [&](int row0, int col) { return row0 < p.out_rows && col < p.n_dim; };
      int fu = first, fc = 0, fk = 0, frow = 0, fcol = 0, fwide = 0;  // the next to fetch: unit and column in it
      bool funit = false;                                            // fk .. fwide are of unit fu
      const auto fetch_next = [&] {
        for (; fu < p.units; fu += step, fc = 0, funit = false) {
          if (!funit) {
            int row, col;
            bool half;
            if (!decode<TALL>(p, kind, fu, fk, row, col, half)) continue;
            fwide = half ? BN / 4 : BN / 2;
            frow = row + BMC * int(rank) + 32 * quarter, fcol = col + side * fwide;
            funit = true;
            bool r = true;
            if (lane == 0) r = wait_ready(ready, ph * a.count + fk, abort_flag, err);
            ok = __all_sync(0xFFFFFFFFu, r);
            if (!ok) {
              fu = p.units;
              return;
            }
          }
          if (fc < fwide && exists(frow, fcol + fc)) break;
        }
        if (fu >= p.units) return;
        const int q = slot ^ ahead;  // ahead is 0 or 1
        if (lane == 0) {
          mbar_arrive_expect_tx_relaxed(&cbar[q], 2 * PART);
          tma_load_2d(from_hi, &cbar[q], mine + q * SLOT, fcol + fc, fk * p.out_rows + frow);
          tma_load_2d(from_lo, &cbar[q], mine + q * SLOT + PART, fcol + fc, fk * p.out_rows + frow);
        }
        flying |= 1 << q;
        ++ahead;
        fc += 32;
      };
      if (kind != kGram) {
        fetch_next();
        if (!last) fetch_next();
      }
      for (int u = first; ok && u < p.units; u += step) {
        int k, row, col;
        bool half;
        if (!decode<TALL>(p, kind, u, k, row, col, half)) {
          if (ew == 0 && lane == 0 && !last) add_release(counters + k);
          continue;
        }
        const int wide = half ? BN / 4 : BN / 2;  // this warp's columns
        const int row0 = row + BMC * int(rank) + 32 * quarter, c0 = col + side * wide, me = row0 + lane;
        // d or e of this lane's row and of the columns
        float own = 0.f, t[4] = {0.f, 0.f, 0.f, 0.f};
        if (kind != kGram) {
          const float *const d = (kind == kPoly ? a.diag : a.e) + int64_t(k) * a.m;
          if ((kind == kPoly || !TALL) && me < a.m) own = __ldcg(d + me);
          if (kind == kPoly || TALL) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c0 + 32 * i + lane < a.m) t[i] = __ldcg(d + c0 + 32 * i + lane);
          }
        }
        // with time to spare the unit before is counted off here, else behind the first chunk
        if (owed && !__all_sync(0xFFFFFFFFu, mbar_test(&tfull[acc], acc_parity))) settle(true);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_parity, abort_flag, err, 0x8u))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t base = tmem_base + (uint32_t(32 * quarter) << 16) + uint32_t(acc * BN + side * wide);
#pragma unroll 1
        for (int c = 0; c < wide; c += 32) {
          const int at = c0 + c;
          if (!exists(row0, at)) break;
          // the slot that the chunk before left: its store has read it by now
          const auto refill = [&] {
            if (ahead < SLOTS) {
              if (lane == 0) bulk_wait_group_read<0>();
              fetch_next();
            }
          };
          if (kind != kGram) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&cbar[slot], (cparity >> slot) & 1u, abort_flag, err, 0x400u))) {
              ok = false;
              break;
            }
            cparity ^= 1u << slot;
            flying &= ~(1 << slot);
            v[lane] = c == 0 ? t[0] : c == 32 ? t[1] : c == 64 ? t[2] : t[3];
          } else if (lane == 0) {
            bulk_wait_group_read<0>();  // the chunk before has left the slots
          }
          __syncwarp();
          uint8_t *const hi_part = mine + (kind == kGram ? 0 : slot * SLOT), *const lo_part = hi_part + PART;
          uint8_t *const staged = mine + (slot ^ 1) * SLOT;  // the chunk before's, free
          const int diagonal = me - at;  // this lane's diagonal element, where the chunk holds it
          float at_diagonal = 0.f;
          if (kind == kUpdate) {
            update_chunk<TALL>(a, base + uint32_t(c), hi_part, lo_part, staged, v, own, me < p.m_dim, early, last, lane);
            if (!last) refill();
            send_chunk(a, &maps.c_hi[~(ph / 3) & 1], &maps.c_lo, hi_part, lo_part, staged, last, lane, k, p.m_dim, p.n_dim,
                       p.out_rows, row0, at);
            if (last) refill();
          } else {
            const float alpha = kind == kGram ? a.x_inv * a.x_inv : a.gram_inv * a.gram_inv;
            const float poly[3] = {fmaf(a.c, own, a.b) * a.gram_inv * a.poly_scale, a.c * a.gram_inv * a.poly_scale,
                                   a.c * alpha * a.poly_scale};
            const bool edge = at == row0;  // the chunk holds a piece of the diagonal
#pragma unroll 1
            for (int j = 0; j < 4; j += 2) {
              uint32_t r[16];
              tmem_ld_32x32b_x16(base + uint32_t(c + 8 * j), r);
              uint32_t h[8], l[8];
              float2 x[8];
              if (kind == kGram) {
                tmem_ld_wait();
                if (edge) gram_row<true>(r, alpha * a.gram_scale, alpha, diagonal - 8 * j, 16, at_diagonal, x);
                else gram_row<false>(r, alpha * a.gram_scale, alpha, 0, 0, at_diagonal, x);
              } else {
                float2 g[8], dj[8];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const uint4 hv = *reinterpret_cast<const uint4 *>(hi_part + piece_at(lane, j + q));
                  const uint4 lv = *reinterpret_cast<const uint4 *>(lo_part + piece_at(lane, j + q));
                  h[4 * q] = hv.x, h[4 * q + 1] = hv.y, h[4 * q + 2] = hv.z, h[4 * q + 3] = hv.w;
                  l[4 * q] = lv.x, l[4 * q + 1] = lv.y, l[4 * q + 2] = lv.z, l[4 * q + 3] = lv.w;
                }
                load16(v + 8 * j, dj);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = add2(unpack2(h[i]), unpack2(l[i]));
                tmem_ld_wait();
                if (edge) poly_row<true>(r, g, dj, poly, alpha, diagonal - 8 * j, 16, at_diagonal, x);
                else poly_row<false>(r, g, dj, poly, alpha, 0, 0, at_diagonal, x);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                h[i] = pack2(x[i].x, x[i].y);
                if (kind == kGram) l[i] = low2(x[i], h[i]);
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                *reinterpret_cast<uint4 *>(hi_part + piece_at(lane, j + q)) = make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
                if (kind == kGram)
                  *reinterpret_cast<uint4 *>(lo_part + piece_at(lane, j + q)) = make_uint4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]);
              }
            }
            if (diagonal >= 0 && diagonal < 32 && me < a.m) {
              if (kind == kGram) a.diag[int64_t(k) * a.m + me] = at_diagonal;
              else a.e[int64_t(k) * a.m + me] = fmaf(a.c, fmaf(own, own, at_diagonal), fmaf(a.b, own, a.a));
            }
            // the chunk, its low part (A'; where the next phase's own tiles are), and its mirror image where no tile
            // computes it: B' leaves that where the low part of A' was
            const bool mirror = at / BMP > row0 / BMP;
            uint8_t *const image = kind == kGram ? lo_part + PART : lo_part;
            if (mirror) {
              __syncwarp();  // every lane has read its low part
              transpose_chunk(hi_part, image, lane);
            }
            if (kind == kPoly) refill();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int to = k * p.out_rows + row0;
              const CUtensorMap *const out = kind == kGram ? &maps.c_gram : &maps.c_poly;
              tma_store_2d(out, hi_part, at, to);
              if (kind == kGram) tma_store_2d(&maps.c_gram_lo, lo_part, at, to);
              if (mirror) tma_store_2d(out, image, row0, k * p.out_rows + at);
              bulk_commit_group();
            }
          }
          if (c == 0) settle(false);
          if (kind != kGram) {
            slot ^= 1;
            --ahead;
          }
        }
        if (!ok) break;
        settle(true);  // where this warp had no chunk
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&tempty[acc], 0));
        if (++acc == 2) {
          acc = 0;
          acc_parity ^= 1u;
        }
        if (!last) owed = counters + k;
      }
      if (!ok || last) break;
      settle(true);
    }
    if (!ok) *abort_flag = 1;
    if (lane == 0) {
      bulk_wait_group_read<0>();  // the slots outlive the stores' reads of them
      for (int s = 0; s < SLOTS; ++s)
        if (flying >> s & 1) drain(&cbar[s], (cparity >> s) & 1u);
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

// --------------------------------------------------------------------------- small Gram matrices

// Matrices whose smaller side fits one tile (128 G: a CTA, or a pair of them): every CTA or pair that shares a matrix
// computes all of A and A^2 by itself, so that A' and B' go from the accumulator to the next product's operand through
// its own shared memory, and an iteration has one exchange, X's, in place of three.
//   GRAM    X's rows (columns, TALL) stream through the ring; one tile in shared memory is both operands, A staying in
//           the accumulator, exact, until B is formed;
//   POLY    A' as the first epilogue left it: each CTA of a pair holds its 128 rows, which are its rows of either operand;
//   UPDATE  B' likewise, against X's tiles: those of this group, `parts` groups a matrix.
// d and e of all rows are traded between the CTAs of a pair.
constexpr int R_STAGE = 128 * BK * 2;  // 128 rows of 64 (or 64 of 128)

struct SmallArgs {
  int count, rows, cols, stand;          // X: its rows in memory
  int parts, groups;                     // CTAs or pairs a matrix, matrices at a time
  int tiles, half;                       // X's tiles; 1: half as wide (TALL: half of the columns each)
  int gram_blocks, poly_blocks;          // blocks of 64 of the contractions
};

struct SmallMaps {
  CUtensorMap x[2], x_tall[2], c_hi[2], c_lo;
};

template <int G>
struct Small {
  static constexpr int N = 128 * G, OP = 2 * G * R_STAGE;  // B' or A': 2 G panels of 64 columns
  static constexpr int STAGES = G == 1 ? 8 : 6;
  static constexpr int VECS = 2 * N * 4;
  static constexpr int SMEM = OP + STAGES * R_STAGE + SMEM_SLOTS + VECS + SMEM_CTRL;  // no room to align it again
};
static_assert(Small<1>::SMEM <= 232448 && Small<2>::SMEM <= 232448, "shared memory per block");

// Where column c (a multiple of 8) of row r of A' or B' lies in the operand: panels of 64 columns in the 128-byte swizzle.
__device__ __forceinline__ int operand_at(int r, int c) { return (c >> 6) * R_STAGE + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4); }

// Waits for a phase of `bar`, with what the other CTA of the pair wrote before its arrivals made visible.
template <int G>
__device__ __forceinline__ bool mbar_wait_group(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned int *err,
                                                unsigned int bit) {
  const bool ok = mbar_wait(bar, parity, abort_flag, err, bit);
  if (G == 2) asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return ok;
}

template <int G, bool TALL>
__global__ void __cluster_dims__(G, 1, 1) __launch_bounds__(kThreads, 1)
    newton_schulz_small_kernel(const __grid_constant__ SmallMaps maps, const __grid_constant__ Args a,
                               const __grid_constant__ SmallArgs s) {
  using S = Small<G>;
  constexpr int N = S::N;
  extern __shared__ __align__(1024) uint8_t smem_at_1024[];  // the host checks that it starts there
  uint8_t *op = smem_at_1024, *ring = op + S::OP, *slots = ring + S::STAGES * R_STAGE;
  float *dvec = reinterpret_cast<float *>(slots + SMEM_SLOTS), *evec = dvec + N;
  uint64_t *full = reinterpret_cast<uint64_t *>(evec + N);
  uint64_t *empty = full + S::STAGES;
  uint64_t *tfull = empty + S::STAGES;
  uint64_t *tempty = tfull + 2;
  uint64_t *op_ready = tempty + 2;   // the even CTA's: A' or B' is in shared memory
  uint64_t *drained = op_ready + 1;
  uint64_t *cfull = drained + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(cfull + SLOTS * kEpilogueWarps);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *ready = abort_flag + 1;
  int *finished = const_cast<int *>(ready + 1);  // warps that have finished their part of an iteration, over all of them
  static_assert((2 * S::STAGES + 6 + SLOTS * kEpilogueWarps) * 8 + 16 <= SMEM_CTRL, "control block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = G == 2 ? cluster_ctarank() : 0;
  const int cluster = int(blockIdx.x) / G, group = cluster / s.parts, part = cluster - group * s.parts;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], G * kEpilogueWarps);
    }
    mbar_init(op_ready, G * kEpilogueWarps);
    mbar_init(drained, 1);
    for (int i = 0; i < SLOTS * kEpilogueWarps; ++i) mbar_init(&cfull[i], 1);
    *abort_flag = 0;
    *ready = 0;
    *finished = 0;
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < S::OP / 16; i += kThreads)  // what lies beside A' and B' stays zero
    reinterpret_cast<uint4 *>(op)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 0 && lane < 7) tma_prefetch_desc(reinterpret_cast<const CUtensorMap *>(&maps) + lane);
  if (warp == 1) {
    if (G == 2) {
      tmem_alloc_pair(tmem_slot, 2 * N);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * N);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (G == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  unsigned int *err = &g_ortho_wait_timeouts;
  // A CTA that has a whole matrix reads nobody else's X: its last warp of an iteration starts the next one, without a round
  // through the counters (84 x 26 32.8 us, with it 36.5).
  const bool alone = G == 1 && s.parts == 1;
  // seq counts this CTA's iterations over all its matrices; `ready` holds the last one that may start
  if (warp == 0) {
    if (lane == 0) {  // -------------------------------------------------- producer: X's tiles, GRAM's then UPDATE's
      int stage = 0;
      uint32_t parity = 0, armed = 0, armed_parity = 0;  // bit s: stage s has been armed, and for which phase
      const uint32_t bars = mapa_shared(full, 0);
      bool ok = true;
      int seq = 0;
      for (int k = group; ok && k < s.count; k += s.groups) {
        const int r0 = k * s.stand;
        for (int it = 0; ok && it < a.steps; ++it, ++seq) {
          if (it > 0 && !(ok = wait_ready(ready, seq, abort_flag, err))) break;
          // blocks of 128 (or 64) indices of a tile from i0 on, 64 of the contraction each; along: it runs along X's rows
          const auto blocks = [&](bool along, int i0, int n, int boxes) {
            const CUtensorMap *const x = along ? &maps.x_tall[it & 1] : &maps.x[it & 1];
            int cx = along ? 0 : i0, cy = along ? r0 + i0 : r0;
            for (int b = 0; b < n; ++b) {
              if (!mbar_wait(&empty[stage], parity ^ 1u, abort_flag, err, 0x1u)) return false;
              if (rank == 0) {
                mbar_arrive_expect_tx_relaxed(&full[stage], along ? G * R_STAGE : G * boxes * BOX);
                armed |= 1u << stage;
                armed_parity = (armed_parity & ~(1u << stage)) | parity << stage;
              }
              uint8_t *const to = ring + stage * R_STAGE;
              for (int i = 0; i < (along ? 1 : boxes); ++i) {
                if (G == 2) tma_load_2d_pair(x, bars + 8 * stage, to + i * BOX, cx + 64 * i, cy);
                else tma_load_2d(x, &full[stage], to + i * BOX, cx + 64 * i, cy);
              }
              if (along) cx += BK;
              else cy += BK;
              if (++stage == S::STAGES) {
                stage = 0;
                parity ^= 1u;
              }
            }
            return true;
          };
          ok = blocks(!TALL, 128 * int(rank), s.gram_blocks, 2);
          const int each = TALL ? 128 : 128 >> s.half;  // of a tile, this CTA's
          for (int t = part; ok && t < s.tiles; t += s.parts)
            ok = blocks(TALL, G * each * (TALL ? t >> s.half : t) + each * int(rank), s.poly_blocks, 2 >> s.half);
        }
      }
      for (int i = 0; i < S::STAGES; ++i)
        if (armed >> i & 1) drain(&full[i], armed_parity >> i & 1);
    }
  } else if (warp == 1) {  // ---------------------------------------------- MMA (the even CTA)
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t parity = 0, acc_parity = 0, op_parity = 0;
      bool ok = true;
      const auto issue = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool more) {
        if (G == 2) mma_f16_pair(d, ad, bd, idesc, more);
        else mma_f16(d, ad, bd, idesc, more);
      };
      const auto commit = [&](uint64_t *bar) {
        if (G == 2) mma_commit_pair(bar, 0x3);
        else mma_commit(bar);
      };
      // One product: `kind`'s contraction into the next accumulator, `wide` columns; rows: of B' before them.
      const auto product = [&](int kind, int blocks, int wide, int rows) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_parity ^ 1u, abort_flag, err, 0x2u))) return false;
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc * N);
        const bool a_mn = kind == kGram && TALL, b_mn = a_mn || (kind == kUpdate && !TALL);
        const uint32_t idesc = idesc_f16_f32(N, wide, a_mn, b_mn);
        const uint32_t da = a_mn ? UK * 128 : UK * 2, db = b_mn ? UK * 128 : UK * 2;
        for (int b = 0; b < blocks; ++b) {
          if (kind != kPoly && !__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], parity, abort_flag, err, 0x4u))) return false;
          tc_fence_after();
          if (elect_one_sync()) {
            const uint32_t x0 = smem_u32(ring + stage * R_STAGE), o0 = smem_u32(op + b * R_STAGE);
            const uint32_t a0 = kind == kGram || (kind == kUpdate && TALL) ? x0 : o0;
            const uint32_t b0 = kind == kGram || (kind == kUpdate && !TALL) ? x0 : o0 + uint32_t(rows) * 128;
#pragma unroll
            for (int i = 0; i < BK / UK; ++i)
              issue(d, sdesc_sw128(a0 + i * da, a_mn ? BOX : 16, 1024), sdesc_sw128(b0 + i * db, b_mn ? BOX : 16, 1024), idesc,
                    b > 0 || i > 0);
            if (kind != kPoly) commit(&empty[stage]);
          }
          __syncwarp();
          if (kind != kPoly && ++stage == S::STAGES) {
            stage = 0;
            parity ^= 1u;
          }
        }
        if (elect_one_sync()) commit(&tfull[acc]);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_parity ^= 1u;
        }
        return true;
      };
      const auto operand = [&] {  // A' or B' is in place
        const bool there = __all_sync(0xFFFFFFFFu, mbar_wait_group<G>(op_ready, op_parity, abort_flag, err, 0x800u));
        op_parity ^= 1u;
        tc_fence_after();
        return there;
      };
      for (int k = group; ok && k < s.count; k += s.groups)
        for (int it = 0; ok && it < a.steps; ++it) {
          ok = product(kGram, s.gram_blocks, N, 0) && operand() && product(kPoly, s.poly_blocks, N, 0) && operand();
          for (int t = part; ok && t < s.tiles; t += s.parts)
            ok = product(kUpdate, s.poly_blocks, N >> s.half, TALL ? 64 * (t & s.half) : 0);
        }
      if (elect_one_sync()) commit(drained);
      __syncwarp();
    }
    if (lane == 0) drain(drained, 0);
  } else if (warp == 3) {
    if (lane == 0) {  // ---------------------------------------------------- X of the iteration before, from all parts
      int seq = 0;
      bool ok = true;
      for (int k = group; ok && k < s.count; k += s.groups)
        for (int it = 0; ok && it < a.steps; ++it, ++seq) {
          if (it == 0 || alone) continue;
          const unsigned int all = unsigned(G * s.parts);
          const uint64_t t0 = globaltimer_ns();
          uint32_t spins = 0;
          while (load_acquire(&a.arrived[k * kMostSteps + it - 1]) < all) {
            if (*abort_flag) ok = false;
            if ((++spins & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
              atomicOr(err, 0x200u);
              ok = false;
            }
            if (!ok) break;
          }
          if (!ok) {
            *abort_flag = 1;
            break;
          }
          fence_proxy_async_global();
          __threadfence_block();
          *ready = seq;
        }
    }
  } else if (warp >= 4) {  // ----------------------------------------------- epilogues (both CTAs)
    const int ew = warp - 4, quarter = warp & 3, side = ew >> 2;
    const int lrow = 32 * quarter + lane, me = 128 * int(rank) + lrow;  // this lane's row of A and B
    uint8_t *const mine = slots + ew * SLOTS * SLOT;
    uint64_t *const cbar = cfull + SLOTS * ew;
    const uint32_t lanes = uint32_t(32 * quarter) << 16;
    const int m_dim = s.rows, n_dim = s.cols;
    int acc = 0, slot = 0, ahead = 0, seq = 0;
    uint32_t acc_parity = 0, cparity = 0;
    int flying = 0;
    bool ok = true;
    const auto result = [&] {  // the next accumulator holds its product
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_parity, abort_flag, err, 0x8u))) return false;
      tc_fence_after();
      return true;
    };
    const auto advance = [&] {
      if (++acc == 2) {
        acc = 0;
        acc_parity ^= 1u;
      }
    };
    const auto release = [&](int which) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&tempty[which], 0));
    };
    // What this warp has written of an operand, and the value of a row's diagonal element for every row's reader in the
    // pair (put: this lane has it).  Who waits for the product of that operand has waited for both.
    const auto hand_over = [&](float *vec, bool put, float value) {
      if (put) {
        vec[me] = value;
        if (G == 2)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(&vec[me], rank ^ 1u)), "f"(value) : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (G == 2) mbar_arrive_cluster(mapa_shared(op_ready, 0));
        else mbar_arrive(op_ready);
      }
    };
    const int first_col = side * (N / 2), first_row = 128 * int(rank) + 32 * quarter;
    const bool exists_row = me < a.m;
    // Whether sixteen columns from c on need more than arithmetic: a piece of the diagonal, the matrix's end.
    const auto edge_at = [&](int c) { return c + 16 > a.m || (c < first_row + 32 && c + 16 > first_row); };
    const auto put_row = [&](int c, const float2 (&x)[8]) {
      if (exists_row) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<uint4 *>(op + operand_at(lrow, c + 8 * q)) =
              make_uint4(pack2(x[4 * q].x, x[4 * q].y), pack2(x[4 * q + 1].x, x[4 * q + 1].y),
                         pack2(x[4 * q + 2].x, x[4 * q + 2].y), pack2(x[4 * q + 3].x, x[4 * q + 3].y));
      }
    };
    for (int k = group; ok && k < s.count; k += s.groups) {
      for (int it = 0; ok && it < a.steps; ++it, ++seq) {
        const bool early = it < a.early, last = it + 1 == a.steps;
        const CUtensorMap *const from = &maps.c_hi[it & 1], *const to = &maps.c_hi[~it & 1];
        // ---- the old X of this group's first chunks, under way while A and B are formed
        if (it > 0) {
          bool r = true;
          if (lane == 0) r = wait_ready(ready, seq, abort_flag, err);
          if (!(ok = __all_sync(0xFFFFFFFFu, r))) break;
        }
        // Half of the columns (TALL) are 64 of each CTA's rows of B'.
        const int wide = (N / 2) >> s.half;  // a warp's columns of a tile
        const auto place = [&](int t, int &row0, int &col) {
          row0 = (TALL ? (t >> s.half) * N : 0) + 128 * int(rank) + 32 * quarter;
          col = TALL ? 64 * (t & s.half) + side * (G == 2 ? N / 2 : wide) : 2 * t * wide + side * wide;
        };
        const auto exists = [&](int row0, int col) { return row0 < s.stand && col < n_dim; };
        int ft = part, fc = 0;  // the next chunk to fetch
        const auto fetch_next = [&] {
          int row0 = 0, col = 0;
          for (; ft < s.tiles; ft += s.parts, fc = 0) {
            place(ft, row0, col);
            if (fc < wide && exists(row0, col + fc)) break;
          }
          if (ft >= s.tiles) return;
          const int q = slot ^ ahead;  // ahead is 0 or 1
          if (lane == 0) {
            mbar_arrive_expect_tx_relaxed(&cbar[q], 2 * PART);
            tma_load_2d(from, &cbar[q], mine + q * SLOT, col + fc, k * s.stand + row0);
            tma_load_2d(&maps.c_lo, &cbar[q], mine + q * SLOT + PART, col + fc, k * s.stand + row0);
          }
          flying |= 1 << q;
          ++ahead;
          fc += 32;
        };
        const auto refill = [&] {  // the slot that the chunk before left: its store has read it by now
          if (ahead < SLOTS) {
            if (lane == 0) bulk_wait_group_read<0>();
            fetch_next();
          }
        };
        fetch_next();
        if (!last) fetch_next();
        // ---- A: the diagonal to d, the rest as fp16
        if (!(ok = result())) break;
        const int gram_acc = acc;
        advance();
        const uint32_t gram = tmem_base + lanes + uint32_t(gram_acc * N + first_col);
        const float g_alpha = a.x_inv * a.x_inv;
        float at_diagonal = 0.f;
        const bool on_diagonal = me >= first_col && me < first_col + N / 2;
        const int cols_here = min(N / 2, a.m - first_col);
#pragma unroll 1
        for (int c = 0; c < cols_here; c += 16) {
          const int at = first_col + c;
          uint32_t r[16];
          tmem_ld_32x32b_x16(gram + uint32_t(c), r);
          tmem_ld_wait();
          float2 x[8];
          if (edge_at(at)) gram_row<true>(r, g_alpha * a.gram_scale, g_alpha, me - at, a.m - at, at_diagonal, x);
          else gram_row<false>(r, g_alpha * a.gram_scale, g_alpha, 0, 0, at_diagonal, x);
          put_row(at, x);
        }
        hand_over(dvec, on_diagonal, at_diagonal);
        // ---- B from A, still exact in its accumulator, and A'^2
        if (!(ok = result())) break;
        const uint32_t square = tmem_base + lanes + uint32_t(acc * N + first_col);
        const float s_alpha = a.gram_inv * a.gram_inv, di = dvec[me];
        const float poly[3] = {fmaf(a.c, di, a.b) * g_alpha * a.poly_scale, a.c * g_alpha * a.poly_scale,
                               a.c * s_alpha * a.poly_scale};
#pragma unroll 1
        for (int c = 0; c < cols_here; c += 16) {
          const int at = first_col + c;
          uint32_t r[16], g[16];
          tmem_ld_32x32b_x16(square + uint32_t(c), r);
          tmem_ld_32x32b_x16(gram + uint32_t(c), g);
          float2 dj[8], gf[8], x[8];
          load16(dvec + at, dj);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) gf[i] = pair_of(g, 2 * i);
          if (edge_at(at)) poly_row<true>(r, gf, dj, poly, s_alpha, me - at, a.m - at, at_diagonal, x);
          else poly_row<false>(r, gf, dj, poly, s_alpha, 0, 0, at_diagonal, x);
          put_row(at, x);
        }
        release(gram_acc);
        release(acc);
        advance();
        hand_over(evec, on_diagonal, fmaf(a.c, fmaf(di, di, at_diagonal), fmaf(a.b, di, a.a)));
        // ---- X of this group's tiles
        for (int t = part; ok && t < s.tiles; t += s.parts) {
          int row0, col;
          place(t, row0, col);
          if (!(ok = result())) break;
          const uint32_t base = tmem_base + lanes + uint32_t(acc * N + side * wide);
          const float own = evec[me];
#pragma unroll 1
          for (int c = 0; c < wide && exists(row0, col + c); c += 32) {
            if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(&cbar[slot], (cparity >> slot) & 1u, abort_flag, err, 0x400u)))) break;
            cparity ^= 1u << slot;
            flying &= ~(1 << slot);
            __syncwarp();
            uint8_t *const hi = mine + slot * SLOT, *const lo = hi + PART;
            uint8_t *const staged = mine + (slot ^ 1) * SLOT;  // the chunk before's, free
            update_chunk<TALL>(a, base + uint32_t(c), hi, lo, staged, &evec[TALL ? col + c : 0], own, row0 + lane < m_dim, early,
                               last, lane);
            if (!last) refill();
            send_chunk(a, to, &maps.c_lo, hi, lo, staged, last, lane, k, m_dim, n_dim, s.stand, row0, col + c);
            if (last) refill();
            slot ^= 1;
            --ahead;
          }
          if (!ok) break;
          release(acc);
          advance();
        }
        if (!ok) break;
        if (!last) {
          if (lane == 0) bulk_wait_all();
          __syncwarp();
          if (lane == 0) {
            __threadfence_block();
            if ((atomicAdd(finished, 1) & (kEpilogueWarps - 1)) == kEpilogueWarps - 1) {
              __threadfence_block();
              if (alone) {
                fence_proxy_async_global();
                __threadfence_block();
                *ready = seq + 1;
              } else {
                add_release(&a.arrived[k * kMostSteps + it]);
              }
            }
          }
        }
      }
    }
    if (!ok) *abort_flag = 1;
    if (lane == 0) {
      bulk_wait_group_read<0>();
      for (int i = 0; i < SLOTS; ++i)
        if (flying >> i & 1) drain(&cbar[i], (cparity >> i) & 1u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (G == 2) cluster_sync();  // neither CTA leaves while the other may still reach its shared memory
  if (warp == 1) {
    tc_fence_after();
    if (G == 2) tmem_dealloc_pair(tmem_base, 2 * N);
    else tmem_dealloc(tmem_base, 2 * N);
  }
}

// --------------------------------------------------------------------------- host

constexpr int64_t kMostElements = (int64_t(1) << 31) - 1, kMostSide = 65536;
constexpr int kMostParts = 1024;

struct Plan {
  int64_t m, n, rows, ldx, planex, grows, ldg, planeg;  // rows, grows: of X and of A with what fills the last block of 64
  int64_t hi[2], lo, gram, gram_lo, poly, diag, e, part, arrived, bytes;  // places in the workspace
};

Plan plan_of(int64_t count, int64_t rows, int64_t cols) {
  Plan p = {};
  p.m = std::min(rows, cols), p.n = std::max(rows, cols);
  // matrices stand on whole blocks of 64 rows: chunks and boxes of one stay within it
  p.rows = (rows + BK - 1) / BK * BK, p.grows = (p.m + BK - 1) / BK * BK;
  p.ldx = (cols + 63) / 64 * 64, p.planex = p.rows * p.ldx;
  p.ldg = p.grows, p.planeg = p.grows * p.ldg;
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
  p.arrived = take(4 * kCounters);
  p.bytes = at;
  return p;
}

struct Schedule {
  float a, b, c;
  int steps;
  float bound;  // on |X|_2 over the operands, from 1
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

// How many clusters of the kernel the device holds at once (a cooperative launch's limit).
template <typename K>
gtp_status clusters_of(K kernel, int size, int smem, std::atomic<int> (&known)[64], const gtp::DeviceInfo &dev,
                       int *clusters) {
  std::atomic<int> &slot = known[dev.device & 63];
  if ((*clusters = slot.load()) > 0) return GTP_OK;
  cudaFuncAttributes f;
  int reserved = 0;
  cudaError_t e = cudaFuncGetAttributes(&f, kernel);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev.device);
  if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "shared memory attributes: %s", cudaGetErrorString(e));
  if (gtp_status s = gtp::check_dynamic_base("orthogonalize", size_t(reserved), f.sharedSizeBytes, 1024))
    return s;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(dev.sm_count / size * size));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  e = cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg);
  if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
  if (*clusters < 1) return gtp::fail(GTP_E_CUDA, "no room for a cluster of %d CTAs", size);
  *clusters = std::min(*clusters, dev.sm_count / size);
  slot.store(*clusters);
  return GTP_OK;
}

// A cooperative launch: the CTAs wait for one another, so all of them run at the same time.
template <typename... KArgs, typename... As>
gtp_status launch_together(void (*kernel)(KArgs...), int ctas, int smem, cudaStream_t st, const As &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return gtp::fail(GTP_E_CUDA, "orthogonalize: %s", cudaGetErrorString(e));
  return gtp::check_launch("orthogonalize");
}

// Tiles of 256 x 256 in whole waves of the pairs, the rest as halves where those fit one wave or less time: a half-wide
// unit takes 0.55 of a whole one's time (a call of 1536 x 2048 217 us; whole tiles alone 268, halves alone 226; 8192 x 2048
// 537, 617, 596; 777 x 1111 155, 218, 155).  Where the other matrices' tiles fill a wave and a half, their phases go into
// one another and whole tiles alone are better (eight of 1536 x 2048 682 us, with halves 690).
void shape(Phase &p, int64_t count, bool symmetric, int64_t k, int pairs) {
  p.tiles_m = (p.m_dim + BMP - 1) / BMP, p.tiles_n = (p.n_dim + BN - 1) / BN;
  p.each = symmetric ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * p.tiles_n;
  p.k_blocks = int((k + BK - 1) / BK);
  const int tiles = int(count) * p.each;
  const auto waves = [&](int units) { return (units + pairs - 1) / pairs; };
  const int whole = tiles / pairs * pairs;
  const double all = waves(tiles), tail = whole / pairs + 0.55 * waves(2 * (tiles - whole)), none = 0.55 * waves(2 * tiles);
  const bool flows = 2 * (count - 1) * p.each >= 3 * pairs;
  p.full = flows || (all <= tail && all <= none) ? tiles : tail <= none ? whole : 0;
  p.units = p.full + 2 * (tiles - p.full);
}

// Matrices of rows x inner fp16, one after another on `stand` rows each.  A box that passes a matrix's last row stays
// in it or reads the next one's: harmless where rows are the product's rows or columns (nobody takes those), and where
// they are the contraction they are zeros.
// box: 32, a chunk of 32 x 32; 64 or 128, as many rows of 64 elements.
gtp_status map_of(CUtensorMap *map, const void *base, int64_t inner, int64_t stand, int64_t ld, int64_t count, uint32_t box) {
  return gtp::encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, uint64_t(inner), uint64_t(count * stand),
                             uint64_t(2 * ld), box == 32 ? 32 : 64, box,
                             box == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// How many iterations scale X's low part by a (see the top): all but the last three.  Singular values spread over four
// decades, the rounding simulated: ten steps 3.0e-3 with seven and 1.2e-2 with two; Gaussian matrices 2.8e-3 with seven
// and 3.2e-3 with two.  Two at least: of five steps, three 8.4e-4 and two 6.5e-4 on a Gaussian matrix.
int early_of(int steps) { return std::max(2, steps - 3); }

// What both kernels need: the iteration's constants and the powers of two that keep every fp16 value in range.
void fill(Args &a, const Schedule &s, const Plan &plan, char *ws) {
  const int xs = 12, gs = 12;
  const double top2 = double(s.bound) * s.bound, poly_top = std::fabs(s.b) * top2 + std::fabs(s.c) * top2 * top2;
  const int ps = std::min(14, 15 - int(std::ceil(std::log2(std::max(poly_top, 1.0)))));
  const auto pow2 = [](int e) { return std::ldexp(1.f, e); };
  a.x_scale = pow2(xs), a.x_inv = pow2(-xs), a.gram_scale = pow2(gs), a.gram_inv = pow2(-gs);
  a.poly_scale = pow2(ps), a.poly_inv = pow2(-ps);
  a.a = s.a, a.b = s.b, a.c = s.c, a.steps = s.steps, a.early = early_of(s.steps), a.m = int(plan.m);
  a.diag = reinterpret_cast<float *>(ws + plan.diag), a.e = reinterpret_cast<float *>(ws + plan.e);
  a.arrived = reinterpret_cast<unsigned int *>(ws + plan.arrived);
}

// The iterations, from X in hi[0] and lo to the last product's output.
template <bool TALL>
gtp_status iterate(Args a, const Plan &plan, char *ws, int64_t count, int64_t rows, int64_t cols, const gtp::DeviceInfo &dev,
                   cudaStream_t st) {
  static std::atomic<int> known[64];
  int pairs = 0;
  a.count = int(count);
  if (gtp_status e = clusters_of(newton_schulz_kernel<TALL>, 2, SMEM_TOTAL, known, dev, &pairs)) return e;
  for (int kind = 0; kind < 3; ++kind) {
    Phase &p = a.phase[kind];
    const bool update = kind == kUpdate;
    p.m_dim = int(update ? rows : plan.m), p.n_dim = int(update ? cols : plan.m);
    p.out_rows = int(update ? plan.rows : plan.grows);
    p.a_rows = int(kind == kGram || (update && TALL) ? plan.rows : plan.grows);
    p.b_rows = int(kind == kGram || (update && !TALL) ? plan.rows : plan.grows);
    shape(p, count, !update, kind == kGram ? plan.n : plan.m, pairs);
  }
  Maps maps;
  const auto x_map = [&](CUtensorMap *m, int64_t at, uint32_t box) {
    return map_of(m, ws + at, cols, plan.rows, plan.ldx, count, box);
  };
  const auto g_map = [&](CUtensorMap *m, int64_t at, uint32_t box) {
    return map_of(m, ws + at, plan.m, plan.grows, plan.ldg, count, box);
  };
  for (const gtp_status e :
       {x_map(&maps.x[0], plan.hi[0], 64), x_map(&maps.x[1], plan.hi[1], 64), x_map(&maps.x_tall[0], plan.hi[0], 128),
        x_map(&maps.x_tall[1], plan.hi[1], 128), g_map(&maps.gram, plan.gram, 64), g_map(&maps.poly, plan.poly, 64),
        g_map(&maps.gram_tall, plan.gram, 128), g_map(&maps.poly_tall, plan.poly, 128), x_map(&maps.c_hi[0], plan.hi[0], 32),
        x_map(&maps.c_hi[1], plan.hi[1], 32), x_map(&maps.c_lo, plan.lo, 32), g_map(&maps.c_gram, plan.gram, 32),
        g_map(&maps.c_gram_lo, plan.gram_lo, 32), g_map(&maps.c_poly, plan.poly, 32)})
    if (e) return e;
  const int used = std::min(pairs, std::max({a.phase[0].units, a.phase[1].units, a.phase[2].units}));
  return launch_together(newton_schulz_kernel<TALL>, 2 * used, SMEM_TOTAL, st, maps, a);
}

template <int G, bool TALL>
gtp_status iterate_small(const Args &a, const Plan &plan, char *ws, int64_t count, int64_t rows, int64_t cols,
                         const gtp::DeviceInfo &dev, cudaStream_t st) {
  static std::atomic<int> known[64];
  int clusters = 0;
  if (gtp_status e = clusters_of(newton_schulz_small_kernel<G, TALL>, G, Small<G>::SMEM, known, dev, &clusters)) return e;
  SmallArgs s = {};
  s.count = int(count), s.rows = int(rows), s.cols = int(cols), s.stand = int(plan.rows);
  s.tiles = int((plan.n + Small<G>::N - 1) / Small<G>::N);
  // tiles half as wide where there are CTAs for twice as many and the second halves exist: finishing a tile is the
  // longest part of an iteration (512 x 256 80 us, whole tiles 93; 128 x 512 50 and 57; eight of 256 x 512 84 and 99)
  s.half = (G == 2 || s.tiles > 1) && 2 * s.tiles * s.count <= clusters && (!TALL || plan.m > 64);
  if (s.half) s.tiles = TALL ? 2 * s.tiles : int((plan.n + Small<G>::N / 2 - 1) / (Small<G>::N / 2));
  s.gram_blocks = int((plan.n + BK - 1) / BK), s.poly_blocks = int((plan.m + BK - 1) / BK);
  s.parts = std::max(1, std::min(s.tiles, clusters / s.count));
  s.groups = std::min(s.count, clusters / s.parts);
  SmallMaps maps;
  const auto x_map = [&](CUtensorMap *m, int64_t at, uint32_t box) {
    return map_of(m, ws + at, cols, plan.rows, plan.ldx, count, box);
  };
  for (const gtp_status e :
       {x_map(&maps.x[0], plan.hi[0], 64), x_map(&maps.x[1], plan.hi[1], 64), x_map(&maps.x_tall[0], plan.hi[0], 128),
        x_map(&maps.x_tall[1], plan.hi[1], 128), x_map(&maps.c_hi[0], plan.hi[0], 32), x_map(&maps.c_hi[1], plan.hi[1], 32),
        x_map(&maps.c_lo, plan.lo, 32)})
    if (e) return e;
  return launch_together(newton_schulz_small_kernel<G, TALL>, G * s.parts * s.groups, Small<G>::SMEM, st, maps, a, s);
}

gtp_status iterate(Args a, const Schedule &s, const Plan &plan, char *ws, int64_t count, int64_t rows, int64_t cols,
                   const gtp::DeviceInfo &dev, cudaStream_t st) {
  fill(a, s, plan, ws);
  const bool tall = rows > cols;
  // a CTA or a pair a matrix's Gram where one tile holds it: 128 x 128 45 us (a pair 61, phases 89), 512 x 256 80 us (phases
  // 103), 256 x 256 71 us (97)
  if (plan.m <= 128)
    return tall ? iterate_small<1, true>(a, plan, ws, count, rows, cols, dev, st)
                : iterate_small<1, false>(a, plan, ws, count, rows, cols, dev, st);
  if (plan.m <= 256)
    return tall ? iterate_small<2, true>(a, plan, ws, count, rows, cols, dev, st)
                : iterate_small<2, false>(a, plan, ws, count, rows, cols, dev, st);
  return tall ? iterate<true>(a, plan, ws, count, rows, cols, dev, st) : iterate<false>(a, plan, ws, count, rows, cols, dev, st);
}

template <typename T, bool VEC, bool STEP>
gtp_status first_of(const Source &s, FirstX f, int64_t count, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const int64_t blocks = (s.items + kPassThreads - 1) / kPassThreads;
  const int64_t fill = std::max<int64_t>(1, int64_t(dev.sm_count) * 8 / count);
  const int64_t most = (blocks + kFlight - 1) / kFlight;
  const dim3 squares(unsigned(std::min<int64_t>({most, fill, kMostParts})), unsigned(count));
  f.parts = int(squares.x);
  if (gtp_status e = gtp::launch_overlapped(squares_kernel<T, VEC, STEP>, squares, kPassThreads, 0, st, "orthogonalize", s, f))
    return e;
  return gtp::launch_overlapped(first_x_kernel<T, VEC, STEP>, dim3(unsigned(std::min(most, fill)), unsigned(count)),
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
  f.arrived = reinterpret_cast<unsigned int *>(ws + plan.arrived);
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
  Args a = {};
  a.dst = dst, a.ld = dst_ld, a.plane = dst_plane, a.dst_f32 = dst_dt == GTP_F32;
  return iterate(a, schedule, plan, ws, count, rows, cols, dev, st);
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
  const float keep = float(1.0 - double(h->lr) * double(h->weight_decay)), rate = float(double(h->lr) * double(h->scale));
  if (!std::isfinite(keep) || !std::isfinite(rate))
    return gtp::fail(GTP_E_ARG, "lr * weight_decay or lr * scale passes fp32");
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
  Args a = {};
  a.step = 1, a.master = master, a.param = static_cast<__nv_bfloat16 *>(param_data);
  a.keep = keep, a.rate = rate;
  for (int64_t k = 0; k < count; ++k) source.offset[k] = a.offset[k] = offsets[k];
  vec = vec && aligned(grad_data, 4 * gs) && aligned(momentum, 16);
  if (gtp_status s = first<true>(source, grad_dt == GTP_F32, vec, first_x(plan, ws), count, rows, cols, dev, st)) return s;
  return iterate(a, schedule, plan, ws, count, rows, cols, dev, st);
}
