// Rotary positions on the heads of a packed projection's output, and their gradient.
//
// Page: "Megatron-LM architecture and source guide" (arganzheng.life), §1 and §4 (the Llama-shape
// model whose QKV projection this rotates between the product and attention).
//
// A pair (a, b) of a head at position p turns by the angle p f_i (f_i the pair's frequency):
//   (a, b) -> (a cos - b sin, a sin + b cos) * scale,
// the gradient by the opposite angle.  The angle is formed in turns as a 64-bit fixed-point
// fraction, p * round(f_i / 2 pi * 2^64) modulo 2^64: the integer product wraps exactly where the
// angle does, so no position, however large, loses any of its fraction (an fp32 product p * f_i is
// off by 4e-3 radians at p = 131072), and the sine is taken of at most half a turn.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "device.h"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

struct Turns {
  uint64_t t[kMaxPairs];
};

struct RotaryArgs {
  const void *src;
  void *dst;
  const void *positions;
  int64_t tokens;
  int64_t src_token, src_group, src_head, dst_token, dst_group, dst_head;
  int64_t pos0, tokens_per_position, positions_per_sequence;
  int32_t heads, group_heads, head_dim, half;  // heads: over all groups
  int32_t interleaved, inverse, positions64;
  float scale;
};

__device__ __forceinline__ int64_t position_of(const RotaryArgs &a, int64_t t) {
  if (a.positions)
    return a.positions64 ? __ldg(static_cast<const int64_t *>(a.positions) + t)
                         : int64_t(__ldg(static_cast<const int32_t *>(a.positions) + t));
  int64_t p = t / a.tokens_per_position;
  if (a.positions_per_sequence) p %= a.positions_per_sequence;
  return a.pos0 + p;
}

__device__ __forceinline__ void turn(uint64_t turns, int64_t pos, const RotaryArgs &a, float &c, float &s) {
  const int64_t f = int64_t(uint64_t(pos) * turns);  // the signed fraction of a turn, times 2^64
  // the top 32 bits decide the angle to 2^-32 of a turn; sincospi takes half turns
  sincospif(float(int32_t(f >> 32)) * 0x1p-31f, &s, &c);
  c *= a.scale;
  s *= a.inverse ? -a.scale : a.scale;
}

__device__ __forceinline__ float load_f32(const float *p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// One thread per pair, or per two elements of the part that keeps its values.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const __grid_constant__ RotaryArgs a, const __grid_constant__ Turns turns, int64_t total) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int slots = (a.head_dim + 1) / 2;
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t th = i / slots;
    const int k = int(i - th * slots);
    const int64_t t = th / a.heads;
    const int h = int(th - t * a.heads), g = h / a.group_heads, gh = h - g * a.group_heads;
    const T *s = static_cast<const T *>(a.src) + t * a.src_token + g * a.src_group + gh * a.src_head;
    T *d = static_cast<T *>(a.dst) + t * a.dst_token + g * a.dst_group + gh * a.dst_head;
    if (k < a.half) {
      const int ia = a.interleaved ? 2 * k : k, ib = a.interleaved ? 2 * k + 1 : k + a.half;
      float c, sn;
      turn(turns.t[k], position_of(a, t), a, c, sn);
      const float x = load_f32(s + ia), y = load_f32(s + ib);
      store_f32(d + ia, x * c - y * sn);
      store_f32(d + ib, x * sn + y * c);
    } else if (s != d) {
      d[2 * k] = s[2 * k];
      if (2 * k + 1 < a.head_dim) d[2 * k + 1] = s[2 * k + 1];
    }
  }
}

}  // namespace

extern "C" gtp_status gtp_rotary_turns(const gtp_rotary_config *cfg, uint64_t *turns, float *scale) {
  gtp::clear_error();
  if (!cfg || !turns || !scale) return gtp::fail(GTP_E_ARG, "null pointer");
  if (cfg->reserved[0] || cfg->reserved[1]) return gtp::fail(GTP_E_ARG, "reserved must be 0");
  const int rot = cfg->rot_dim;
  if (rot < 2 || rot % 2 || rot > 2 * kMaxPairs)
    return gtp::fail(GTP_E_SHAPE, "rot_dim must be even, 2 to %d", 2 * kMaxPairs);
  if (!(cfg->base > 1.0) || !std::isfinite(cfg->base)) return gtp::fail(GTP_E_ARG, "base must be above 1");
  if (cfg->scaling < GTP_ROTARY_UNSCALED || cfg->scaling > GTP_ROTARY_RAMP)
    return gtp::fail(GTP_E_ARG, "unknown scaling %d", cfg->scaling);
  const bool scaled = cfg->scaling != GTP_ROTARY_UNSCALED;
  const bool banded = cfg->scaling == GTP_ROTARY_BANDS || cfg->scaling == GTP_ROTARY_RAMP;
  if (scaled && (!(cfg->factor >= 1.0) || !std::isfinite(cfg->factor)))
    return gtp::fail(GTP_E_ARG, "factor must be 1 or more");
  if (cfg->scaling == GTP_ROTARY_BASE && rot == 2) return gtp::fail(GTP_E_SHAPE, "base scaling needs rot_dim above 2");
  if (banded && (cfg->context < 1 || !(cfg->low_turns > 0.0) || !(cfg->high_turns > cfg->low_turns) ||
                 !std::isfinite(cfg->high_turns)))
    return gtp::fail(GTP_E_ARG, "context must be positive and 0 < low_turns < high_turns");
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double base = cfg->base;
  if (cfg->scaling == GTP_ROTARY_BASE) base *= std::pow(cfg->factor, double(rot) / double(rot - 2));
  // GTP_ROTARY_RAMP blends over pair indices, between the (fractional) indices whose frequencies make
  // high_turns and low_turns turns over the context, rounded outwards to whole pairs
  double first = 0, last = 0;
  if (cfg->scaling == GTP_ROTARY_RAMP) {
    const auto index = [&](double n) {
      return rot * std::log(double(cfg->context) / (n * kTwoPi)) / (2 * std::log(base));
    };
    first = std::max(0.0, std::floor(index(cfg->high_turns)));
    last = std::min(double(rot - 1), std::ceil(index(cfg->low_turns)));
    if (last <= first) last = first + 0.001;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (cfg->scaling == GTP_ROTARY_LINEAR) f /= cfg->factor;
    if (banded) {
      double keep;  // the share of the unscaled frequency
      if (cfg->scaling == GTP_ROTARY_BANDS)
        keep = (double(cfg->context) * f / kTwoPi - cfg->low_turns) / (cfg->high_turns - cfg->low_turns);
      else
        keep = 1.0 - (i - first) / (last - first);
      keep = std::min(1.0, std::max(0.0, keep));
      f = keep * f + (1.0 - keep) * f / cfg->factor;
    }
    turns[i] = uint64_t(std::nearbyint(f / kTwoPi * 0x1p64));  // f <= 1, so below 2^62
  }
  *scale = cfg->scaling == GTP_ROTARY_RAMP ? float(0.1 * std::log(cfg->factor) + 1.0) : 1.f;
  return GTP_OK;
}

extern "C" gtp_status gtp_rotary(const gtp_rotary_desc *d, gtp_stream stream) {
  gtp::clear_error();
  if (!d) return gtp::fail(GTP_E_ARG, "null descriptor");
  if (d->dtype != GTP_F32 && d->dtype != GTP_BF16) return gtp::fail(GTP_E_DTYPE, "dtype must be F32 or BF16");
  if (d->reserved || d->interleaved < 0 || d->interleaved > 1 || d->inverse < 0 || d->inverse > 1 ||
      d->positions64 < 0 || d->positions64 > 1)
    return gtp::fail(GTP_E_ARG, "flags must be 0 or 1 and reserved 0");
  if (d->tokens < 0 || d->groups < 0 || d->heads < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (d->head_dim < 1 || d->head_dim > 65536) return gtp::fail(GTP_E_SHAPE, "head_dim must be 1 to 65536");
  if (d->rot_dim < 2 || d->rot_dim % 2 || d->rot_dim > 2 * kMaxPairs || d->rot_dim > d->head_dim)
    return gtp::fail(GTP_E_SHAPE, "rot_dim must be even, 2 to %d and at most head_dim", 2 * kMaxPairs);
  if (d->tokens > (int64_t(1) << 32) || int64_t(d->groups) * d->heads > (1 << 20))
    return gtp::fail(GTP_E_SHAPE, "more than 2^32 tokens or 2^20 heads");
  if (!d->turns) return gtp::fail(GTP_E_ARG, "null turns");
  if (!std::isfinite(d->scale)) return gtp::fail(GTP_E_ARG, "scale must be finite");
  if (d->tokens_per_position < 1 || d->positions_per_sequence < 0)
    return gtp::fail(GTP_E_ARG, "tokens_per_position must be positive and positions_per_sequence 0 or more");
  const int64_t strides[6] = {d->src_token, d->src_group, d->src_head, d->dst_token, d->dst_group, d->dst_head};
  for (int64_t s : strides)
    if (s < 0 || s > (int64_t(1) << 40)) return gtp::fail(GTP_E_ARG, "a stride is negative or above 2^40");
  if (d->tokens == 0 || d->groups == 0 || d->heads == 0) return GTP_OK;
  if (!d->src || !d->dst) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t es = d->dtype == GTP_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(d->src) | reinterpret_cast<uintptr_t>(d->dst)) & uintptr_t(es - 1))
    return gtp::fail(GTP_E_ALIGN, "src and dst must be aligned to their elements");
  if (reinterpret_cast<uintptr_t>(d->positions) & (d->positions64 ? 7u : 3u))
    return gtp::fail(GTP_E_ALIGN, "positions must be aligned to its elements");
  // every two heads of dst are apart: in some order each stride covers what the smaller ones span
  struct Dim {
    int64_t stride, n;
  } dims[3] = {{d->dst_token, d->tokens}, {d->dst_group, d->groups}, {d->dst_head, d->heads}};
  std::sort(dims, dims + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
  int64_t span = d->head_dim;
  for (const Dim &m : dims) {
    if (m.n == 1) continue;
    if (m.stride < span) return gtp::fail(GTP_E_ARG, "the heads of dst overlap");
    if (m.stride > (int64_t(1) << 50) / m.n) return gtp::fail(GTP_E_SHAPE, "dst spans more than 2^50 elements");
    span += (m.n - 1) * m.stride;
  }
  if (d->src_token > (int64_t(1) << 50) / d->tokens) return gtp::fail(GTP_E_SHAPE, "src spans more than 2^50 elements");
  const int64_t src_span =
      (d->tokens - 1) * d->src_token + (d->groups - 1) * d->src_group + (d->heads - 1) * d->src_head + d->head_dim;
  const gtp::ByteRange in = gtp::byte_range(d->src, src_span * es), out = gtp::byte_range(d->dst, span * es);
  const bool in_place = d->src == d->dst && (d->tokens == 1 || d->src_token == d->dst_token) &&
                        (d->groups == 1 || d->src_group == d->dst_group) &&
                        (d->heads == 1 || d->src_head == d->dst_head);
  if (!in_place && gtp::overlap(in, out))
    return gtp::fail(GTP_E_ARG, "src and dst overlap and are not the same heads in place");
  if (d->positions && gtp::overlap(out, gtp::byte_range(d->positions, d->tokens * (d->positions64 ? 8 : 4))))
    return gtp::fail(GTP_E_ARG, "dst overlaps positions");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  RotaryArgs a = {};
  a.src = d->src;
  a.dst = d->dst;
  a.positions = d->positions;
  a.tokens = d->tokens;
  a.src_token = d->src_token, a.src_group = d->src_group, a.src_head = d->src_head;
  a.dst_token = d->dst_token, a.dst_group = d->dst_group, a.dst_head = d->dst_head;
  a.pos0 = d->pos0;
  a.tokens_per_position = d->tokens_per_position;
  a.positions_per_sequence = d->positions_per_sequence;
  a.group_heads = d->heads;
  a.heads = d->groups * d->heads;
  a.head_dim = d->head_dim;
  a.half = d->rot_dim / 2;
  a.interleaved = d->interleaved, a.inverse = d->inverse, a.positions64 = d->positions64;
  a.scale = d->scale;
  Turns turns = {};
  std::copy(d->turns, d->turns + a.half, turns.t);
  const int64_t total = d->tokens * a.heads * ((d->head_dim + 1) / 2);
  const int grid = int(std::min<int64_t>((total + kThreads - 1) / kThreads, int64_t(dev.sm_count) * 8));
  cudaStream_t st = gtp::as_stream(stream);
  if (d->dtype == GTP_F32) return gtp::launch_overlapped(rotary_kernel<float>, grid, kThreads, 0, st, "rotary", a, turns, total);
  return gtp::launch_overlapped(rotary_kernel<__nv_bfloat16>, grid, kThreads, 0, st, "rotary", a, turns, total);
}
