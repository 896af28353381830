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

#include "byte_range.h"
#include "device.h"
#include "fastdiv.cuh"
#include "philox.cuh"
#include "sm100_ptx.cuh"
#include "wide.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kThreads = 256;

struct DropArgs {
  const void *x, *residual;
  void *out;
  int64_t rows, cols, x_ld, residual_ld, out_ld;
  int64_t row0;  // rows before these in the call (a later launch of one call)
  uint32_t threshold;
  float scale;
  gtp::RngArgs rng;
};

// Eight consecutive elements on 16 bytes (bf16) or 32 (fp32), as they lie in memory: loads in flight hold no
// more registers than bytes.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  uint32_t a[8];
  __device__ __forceinline__ void load(const float *p) { gtp::load_32b(p, a); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(a[i]);
  }
  static __device__ __forceinline__ void store(float *p, const float (&x)[8]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    gtp::store_32b(p, w);
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);  // bf16 -> fp32 is exact
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};

// Element k of a group is kept where its 16 bits reach the threshold: the upper half of a word compares
// as the whole word against threshold << 16 (what lies below cannot carry), the lower one shifted up.
// threshold 65536 (p = 1) has no such word and is handled as `none`.
struct Mask {
  uint32_t w[4], cut;
  bool none;
  __device__ __forceinline__ Mask(const DropArgs &a, uint64_t offset, int64_t g, int64_t row) {
    const uint4 d = gtp::philox(a.rng, uint32_t(g) | (gtp::kStreamDropout << 30), uint32_t(row),
                                uint32_t(offset), uint32_t(offset >> 32));
    w[0] = d.x, w[1] = d.y, w[2] = d.z, w[3] = d.w;
    cut = a.threshold << 16;
    none = a.threshold > 65535u;
  }
  __device__ __forceinline__ bool keep(int k) const {
    return (k & 1 ? w[k >> 1] : w[k >> 1] << 16) >= cut && !none;
  }
};

__device__ __forceinline__ uint64_t mul2(float a, float b, float s) {
  uint64_t r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %3};\n\tmul.rn.f32x2 %0, x, y;\n\t}"
      : "=l"(r)
      : "f"(a), "f"(b), "f"(s));
  return r;
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// A thread owns one group of eight columns (one generator call) in ROWS rows at a time, whose loads
// are in flight together; blocks are blockDim.x groups wide and step down the rows.  Every row of every
// array starts on 16 bytes and holds whole groups.
//
// How many rows, and blocks an SM (the grid, and what the registers are held to), measured on 2048 columns:
// bf16 onto a bf16 residual (8192 rows) 17.1 us with 1 row and 8 blocks against 18.3 with 6 and 20-23 with
// 2 or 4 rows; bf16 alone (32768 rows), which the generator bounds, 44.9 us with 4 rows and 4 blocks against
// 45.5-47.7; fp32 to bf16 59.6 us with 2 rows and 4 blocks against 62-74; bf16 onto fp32 (8192 rows) 26.7 us
// with 2 rows and 3 blocks against 30 with the 2 that unbounded registers leave.  Where fp32 moves, a grid of
// up to 16 blocks an SM (26.3 us against 28-30 with 3 to 5): the hardware balances it.
template <typename TI, typename TO, bool RES>
struct Shape {
  static constexpr bool NARROW = sizeof(TI) == 2 && sizeof(TO) == 2;
  static constexpr int ROWS = !NARROW ? 2 : RES ? 1 : 4;
  static constexpr int MIN_BLOCKS = !RES ? 4 : NARROW ? 8 : 3;
  static constexpr int BLOCKS = !NARROW ? 16 : MIN_BLOCKS;
};

template <typename TI, typename TO, bool RES>
__global__ void __launch_bounds__(kThreads, Shape<TI, TO, RES>::MIN_BLOCKS)
    dropout_kernel(const __grid_constant__ DropArgs a) {
  constexpr int N = Shape<TI, TO, RES>::ROWS;
  gtp::ptx::allow_dependents();
  const int64_t g = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  gtp::ptx::wait_prior_grid();
  if (8 * g >= a.cols) return;
  const uint64_t offset = gtp::rng_offset(a.rng);
  const int64_t step = int64_t(gridDim.y) * blockDim.y;
  for (int64_t r0 = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; r0 < a.rows; r0 += N * step) {
    Eight<TI> x[N];
    Eight<TO> res[RES ? N : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step;
      if (row < a.rows) {
        x[i].load(static_cast<const TI *>(a.x) + row * a.x_ld + 8 * g);
        if (RES) res[i].load(static_cast<const TO *>(a.residual) + row * a.residual_ld + 8 * g);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step;
      if (row < a.rows) {
        const Mask m(a, offset, g, row);
        float v[8], y[8];
        x[i].get(v);
        if (RES) {
          res[i].get(y);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (m.keep(k)) y[k] = fmaf(v[k], a.scale, y[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; k += 2) {  // two products an instruction
            const uint64_t z = mul2(v[k], v[k + 1], a.scale);
            y[k] = m.keep(k) ? __uint_as_float(uint32_t(z)) : 0.f;
            y[k + 1] = m.keep(k + 1) ? __uint_as_float(uint32_t(z >> 32)) : 0.f;
          }
        }
        Eight<TO>::store(static_cast<TO *>(a.out) + row * a.out_ld + 8 * g, y);
      }
    }
  }
}

// Rows that start anywhere (odd lengths, strides and bases).  A lane still makes one generator call, for
// group v of a row, and keeps its mask as eight bits; but the eight elements it moves are those from
// column head + 8 v on, where head columns lie before the row's first 16-byte place: its own last
// 8 - head and the first `head` of group v + 1, whose mask the lane above holds.  Items (row, v) run
// over each row's groups one after the other, narrow rows side by side in a warp; the last lane of a
// warp only draws (1/32 of the calls).  The up to 7 columns before and after a row's vectors go element
// by element, a thread each, in the blocks after the others.
//
// That needs one `head` for all arrays of a row, i.e. rows of like length one after another: the
// ordinary odd case.  Arrays that lie differently take dropout_elements_kernel.
//
// [4000, 3001] fp32 onto fp32 22.2 us (96 % of a copy's rate), bf16 alone 12.2 (58 %: the calls, a lane in 32 of
// which is lost, and the mask's way through bits), [16384, 1001] bf16 onto bf16 18.4 (79 %).
struct Shifted {
  int32_t items;        // groups of all rows
  int32_t vector_blocks;
  gtp::FastDiv by_groups;
  int32_t groups;       // of a row, one more than it has whole vectors at most
};

template <typename TI, typename TO, bool RES>
__device__ __forceinline__ void one_element(const DropArgs &a, uint64_t offset, int64_t row, int64_t j) {
  const Mask m(a, offset, j >> 3, row + a.row0);
  const int k = int(j & 7);
  const uint32_t word = k < 2 ? m.w[0] : k < 4 ? m.w[1] : k < 6 ? m.w[2] : m.w[3];
  const bool keep = (k & 1 ? word : word << 16) >= m.cut && !m.none;
  const float x = load1(static_cast<const TI *>(a.x) + row * a.x_ld + j);
  float y = RES ? load1(static_cast<const TO *>(a.residual) + row * a.residual_ld + j) : 0.f;
  if (keep) y = RES ? fmaf(x, a.scale, y) : x * a.scale;
  store1(static_cast<TO *>(a.out) + row * a.out_ld + j, y);
}

template <typename TO>
__device__ __forceinline__ int head_of(const DropArgs &a, int64_t row) {
  const uintptr_t first = reinterpret_cast<uintptr_t>(static_cast<const TO *>(a.out) + row * a.out_ld);
  return int((0u - uint32_t(first / sizeof(TO))) & 7u);
}

// Items a thread, loaded together; with 1 / 2 / 3: bf16 alone [16384, 3001] 48.1 / 45.8 / 43.2 us, bf16 onto
// bf16 [16384, 1001] 19.3 / 18.4 / 18.7, fp32 to bf16 [8001, 3001] 24.4 / 23.3 / 23.9, bf16 onto fp32
// [8001, 3001] 36.1 / 36.2 / 36.7 (98 % of a copy's rate).
template <typename TI, typename TO, bool RES>
constexpr int kShiftedItems = sizeof(TI) + sizeof(TO) > 4 ? (RES ? 1 : 2) : RES ? 2 : 3;

template <typename TI, typename TO, bool RES>
__global__ void __launch_bounds__(kThreads)
    dropout_shifted_kernel(const __grid_constant__ DropArgs a, const __grid_constant__ Shifted s) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const uint64_t offset = gtp::rng_offset(a.rng);
  if (int(blockIdx.x) >= s.vector_blocks) {  // the ends: 16 threads a row
    const int64_t i = int64_t(blockIdx.x - s.vector_blocks) * kThreads + threadIdx.x, row = i >> 4;
    if (row >= a.rows) return;
    const int e = int(i & 15);
    const int64_t head = min(int64_t(head_of<TO>(a, row)), a.cols), tail = head + (a.cols - head) / 8 * 8;
    const int64_t j = e < 8 ? e : tail + e - 8;
    if (e < 8 ? j < head : j < a.cols) one_element<TI, TO, RES>(a, offset, row, j);
    return;
  }
  constexpr int N = kShiftedItems<TI, TO, RES>;
  const int lane = threadIdx.x & 31;
  const int first = (int(blockIdx.x) * (kThreads / 32) + int(threadIdx.x >> 5)) * N * 31 + lane;
  Eight<TI> x[N];
  Eight<TO> res[RES ? N : 1];
  int row[N], v[N], head[N];
  bool whole[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int item = min(first + 31 * i, s.items - 1);
    row[i] = gtp::fast_div(item, s.by_groups);
    v[i] = item - row[i] * s.groups;
    head[i] = head_of<TO>(a, row[i]);
    const int64_t j = head[i] + 8 * int64_t(v[i]);
    whole[i] = lane < 31 && first + 31 * i < s.items && j + 8 <= a.cols;
    if (whole[i]) {
      x[i].load(static_cast<const TI *>(a.x) + row[i] * a.x_ld + j);
      if (RES) res[i].load(static_cast<const TO *>(a.residual) + row[i] * a.residual_ld + j);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Mask m(a, offset, v[i], row[i] + a.row0);
    uint32_t keep = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) keep |= (m.keep(k) ? 1u : 0u) << k;
    // where head > 0 the vector reaches into group v + 1 of the same row, which exists
    keep = (keep | __shfl_down_sync(0xFFFFFFFFu, keep, 1) << 8) >> head[i];
    if (!whole[i]) continue;
    float f[8], y[8];
    x[i].get(f);
    if (RES) res[i].get(y);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!RES) y[k] = 0.f;
      if (keep >> k & 1) y[k] = RES ? fmaf(f[k], a.scale, y[k]) : f[k] * a.scale;
    }
    Eight<TO>::store(static_cast<TO *>(a.out) + row[i] * a.out_ld + head[i] + 8 * int64_t(v[i]), y);
  }
}

// Arrays that lie differently: a thread a group, element by element.  [8192, 2048] bf16 42.3 us (23 % of a copy's rate),
// fp32 66.7 (30 %): neighbouring threads' elements are 16 or 32 bytes apart, eight accesses for each vector of the others.
template <typename TI, typename TO, bool RES>
__global__ void __launch_bounds__(kThreads)
    dropout_elements_kernel(const __grid_constant__ DropArgs a, const __grid_constant__ Shifted s) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const uint64_t offset = gtp::rng_offset(a.rng);
  const int64_t item = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (item >= s.items) return;
  const int row32 = gtp::fast_div(int(item), s.by_groups), v = int(item) - row32 * s.groups;
  const int64_t row = row32;
  const Mask m(a, offset, v, row + a.row0);
  const TI *x = static_cast<const TI *>(a.x) + row * a.x_ld;
  const TO *res = static_cast<const TO *>(a.residual) + (RES ? row * a.residual_ld : 0);
  TO *out = static_cast<TO *>(a.out) + row * a.out_ld;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t j = 8 * int64_t(v) + k;
    if (j < a.cols) {
      float y = RES ? load1(res + j) : 0.f;
      if (m.keep(k)) y = RES ? fmaf(load1(x + j), a.scale, y) : load1(x + j) * a.scale;
      store1(out + j, y);
    }
  }
}

template <typename TI, typename TO, bool RES>
gtp_status launch(DropArgs a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  // the arrays' rows start the same number of elements past 16 bytes: their strides agree modulo 8
  // elements and their first elements do
  const auto at = [](const void *p, size_t es) { return (reinterpret_cast<uintptr_t>(p) / es) & 7u; };
  const auto like_out = [&](const void *p, int64_t ld, size_t es) {
    return at(p, es) == at(a.out, sizeof(TO)) && (a.rows == 1 || (ld - a.out_ld) % 8 == 0);
  };
  const bool same = like_out(a.x, a.x_ld, sizeof(TI)) && (!RES || like_out(a.residual, a.residual_ld, sizeof(TO)));
  const bool aligned = same && at(a.out, sizeof(TO)) == 0 && (a.rows == 1 || a.out_ld % 8 == 0) && a.cols % 8 == 0;
  const int64_t groups = (a.cols + 7) / 8;
  if (aligned) {
    using S = Shape<TI, TO, RES>;
    int tx = 1;
    while (tx < kThreads && tx < groups) tx *= 2;
    const dim3 block(tx, kThreads / tx);
    const int64_t per = block.y * S::ROWS, gx = (groups + tx - 1) / tx;
    const int64_t fill = std::max<int64_t>(1, (int64_t(dev.sm_count) * S::BLOCKS + gx / 2) / gx);
    const dim3 grid(unsigned(gx), unsigned(std::min<int64_t>({(a.rows + per - 1) / per, fill, 65535})));
    return gtp::launch_overlapped(dropout_kernel<TI, TO, RES>, grid, block, 0, st, "dropout", a);
  }
  // items are counted in 31 bits: more than 2^30 groups go in several launches
  const int64_t rows = a.rows, most = std::max<int64_t>(1, (int64_t(1) << 30) / groups);
  const char *x = static_cast<const char *>(a.x), *res = static_cast<const char *>(a.residual);
  char *out = static_cast<char *>(a.out);
  for (int64_t r = 0; r < rows; r += most) {
    a.row0 = r;
    a.rows = std::min(most, rows - r);
    a.x = x + r * a.x_ld * int64_t(sizeof(TI));
    a.residual = RES ? res + r * a.residual_ld * int64_t(sizeof(TO)) : nullptr;
    a.out = out + r * a.out_ld * int64_t(sizeof(TO));
    Shifted s;
    s.groups = int32_t(groups);
    s.by_groups = gtp::make_fastdiv(s.groups);
    s.items = int32_t(a.rows * groups);
    const int64_t a_block = 31 * (kThreads / 32) * kShiftedItems<TI, TO, RES>;
    s.vector_blocks = int32_t((s.items + a_block - 1) / a_block);
    const int64_t end_blocks = (a.rows * 16 + kThreads - 1) / kThreads;
    const gtp_status e =
        same ? gtp::launch_overlapped(dropout_shifted_kernel<TI, TO, RES>, unsigned(s.vector_blocks + end_blocks), kThreads,
                                      0, st, "dropout", a, s)
             : gtp::launch_overlapped(dropout_elements_kernel<TI, TO, RES>, unsigned((s.items + kThreads - 1) / kThreads),
                                      kThreads, 0, st, "dropout", a, s);
    if (e) return e;
  }
  return GTP_OK;
}

template <typename TI, typename TO>
gtp_status launch(const DropArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  return a.residual ? launch<TI, TO, true>(a, dev, st) : launch<TI, TO, false>(a, dev, st);
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
  if (rows > 1 && std::max({x_ld, out_ld, residual ? residual_ld : 0}) > (int64_t(1) << 50) / rows)
    return gtp::fail(GTP_E_SHAPE, "an array spans more than 2^50 elements");
  if (!x || !out) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t xs = x_dt == GTP_F32 ? 4 : 2, os = out_dt == GTP_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) & uintptr_t(xs - 1)) ||
      ((reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(out)) & uintptr_t(os - 1)))
    return gtp::fail(GTP_E_ALIGN, "arrays must be aligned to their elements");
  if (rows == 1) x_ld = residual_ld = out_ld = cols;
  const auto runs = [&](const void *p, int64_t ld, int64_t es) {
    return gtp::Runs{reinterpret_cast<uintptr_t>(p), cols * es, {{ld * es, rows}, {0, 1}, {0, 1}}};
  };
  const gtp::Runs o = runs(out, out_ld, os);
  // in place is fine where every element is read and written by one thread: same start, stride, type; no thread
  // touches anything between the rows, so columns of one buffer may stand side by side
  if (!(x == out && x_dt == out_dt && x_ld == out_ld) && gtp::overlap(o, runs(x, x_ld, xs)))
    return gtp::fail(GTP_E_ARG, "out overlaps the input and is not it");
  if (residual && !(residual == out && residual_ld == out_ld) && gtp::overlap(o, runs(residual, residual_ld, os)))
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
