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

#include "byte_range.h"
#include "device.h"
#include "fastdiv.cuh"
#include "sm100_ptx.cuh"
#include "wide.cuh"

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
  int32_t inverse, positions64, block_tokens, copy;  // copy: the part that keeps its values is written
  int32_t chunks, units;                             // chunks of a head and of a token
  gtp::FastDiv by_half, by_units, by_chunks, by_group;
  float scale;
};

// Positions are read by ordinary loads: the kernel before this one may have written them.
__device__ __forceinline__ int64_t position_of(const RotaryArgs &a, int64_t t) {
  if (a.positions)
    return a.positions64 ? __ldca(static_cast<const long long *>(a.positions) + t)
                         : int64_t(__ldca(static_cast<const int32_t *>(a.positions) + t));
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

// A chunk of a head is 8 pairs: two runs of 8 elements half a rotation apart, or 16 in a row.  With
// heads on whole vectors of 8 elements (VEC; 16 bytes, fp32 32) a chunk moves in those, else element by
// element, a pair a chunk.
template <typename T>
struct Run;
template <>
struct Run<float> {
  uint32_t v[8];
  __device__ __forceinline__ void load(const float *p) { gtp::load_32b(p, v); }
  __device__ __forceinline__ void store(float *p) const { gtp::store_32b(p, v); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(x[i]);
  }
};
template <>
struct Run<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { __stcs(reinterpret_cast<uint4 *>(p), v); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);  // bf16 -> fp32 is exact
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float load_f32(const float *p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

struct Head {
  int64_t src, dst;
};

__device__ __forceinline__ Head head_of(const RotaryArgs &a, int64_t t, int h) {
  const int g = gtp::fast_div(h, a.by_group), gh = h - g * a.group_heads;
  return {t * a.src_token + g * a.src_group + gh * a.src_head, t * a.dst_token + g * a.dst_group + gh * a.dst_head};
}

// One chunk of a head: its two runs, loaded, turned by 8 (cosine, sine) pairs, stored.
template <typename T, bool IL>
struct Chunk {
  Run<T> u, v;
  T *a, *b;
  const float2 *w;
  int pitch;
  __device__ __forceinline__ void load(const RotaryArgs &g, const float2 *cs, int64_t t0, int i) {
    const int t = gtp::fast_div(i, g.by_units), r = i - t * g.units;
    const int h = gtp::fast_div(r, g.by_chunks), c = r - h * g.chunks;
    const Head at = head_of(g, t0 + t, h);
    const int ia = IL ? 16 * c : 8 * c, ib = IL ? ia + 8 : ia + g.half;
    const T *src = static_cast<const T *>(g.src) + at.src;
    u.load(src + ia);
    v.load(src + ib);
    a = static_cast<T *>(g.dst) + at.dst + ia;
    b = static_cast<T *>(g.dst) + at.dst + ib;
    w = cs + t * g.half + 2 * c;
    pitch = 2 * g.chunks;
  }
  __device__ __forceinline__ void turn_and_store() {
    float x[8], y[8];
    u.get(x);
    v.get(y);
    float4 m2;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if ((k & 1) == 0) m2 = *reinterpret_cast<const float4 *>(w + (k >> 1) * pitch);
      // interleaved: pairs 0-3 of the chunk lie in the first run, 4-7 in the second
      float &p = IL ? (k < 4 ? x[2 * k] : y[2 * k - 8]) : x[k];
      float &q = IL ? (k < 4 ? x[2 * k + 1] : y[2 * k - 7]) : y[k];
      const float2 m = k & 1 ? make_float2(m2.z, m2.w) : make_float2(m2.x, m2.y);
      const float np = p * m.x - q * m.y, nq = p * m.y + q * m.x;
      p = np;
      q = nq;
    }
    u.set(x);
    v.set(y);
    u.store(a);
    v.store(b);
  }
};

// A block owns a.block_tokens tokens: it forms each (token, pair)'s cosine and sine once, in shared
// memory, and every head of the token uses them.  The first chunks' loads go out before that, so the
// sines run under their latency.
//
// Chunks a thread (all loaded ahead) and blocks an SM, measured: bf16 (32768 tokens of 20 heads of 128) 49.3 us
// with 2 and 5 against 56.7 (2, unbounded registers), 51.9 (1 ahead, 6) and 63.1 (1 and 6); fp32 (32769
// tokens of 20 heads, 64 of 128 elements turned) 101.7 us with 1 and 6 against 110.2 (2 and 5).
//
// The bytes bound it: 6.8 TB/s on both of these (49.3 and 97.7 us since rows of 32 bytes), the rate of a copy.
// 8192 tokens of 20 heads of 64 (the packed QKV product of a microbatch) take 9.1 us, 4.6 TB/s: the ramp and the
// drain of one wave.  Blocks that stay and load ahead of the sines were slower there.  Heads off whole vectors (8192
// tokens of 20 heads of 65, 64 turned), element by element, take 30.5 us in bf16 (21 % of a copy's rate) and 32.4 in fp32 (39 %).
template <typename T>
struct Shape {
  static constexpr int CHUNKS = sizeof(T) == 2 ? 2 : 1;
  static constexpr int MIN_BLOCKS = sizeof(T) == 2 ? 5 : 6;
};

template <typename T, bool VEC, bool IL>
__global__ void __launch_bounds__(kThreads, Shape<T>::MIN_BLOCKS)
    rotary_kernel(const __grid_constant__ RotaryArgs a, const __grid_constant__ Turns turns) {
  extern __shared__ __align__(16) float2 cs[];  // [block_tokens][half]
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int64_t t0 = int64_t(blockIdx.x) * a.block_tokens;
  const int nt = int(min(int64_t(a.block_tokens), a.tokens - t0));
  constexpr int P = VEC ? 8 : 1, N = Shape<T>::CHUNKS;
  const int all = nt * a.units;
  Chunk<T, IL> ahead[N];
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (int(threadIdx.x) + k * kThreads < all) ahead[k].load(a, cs, t0, threadIdx.x + k * kThreads);
  }
  for (int i = threadIdx.x; i < nt * a.half; i += kThreads) {
    const int t = gtp::fast_div(i, a.by_half), k = i - t * a.half;
    // a chunk's eight pairs, two by two, one run of all chunks after the other: lanes on neighbouring
    // chunks then read neighbouring 16 bytes
    const int at = VEC ? t * a.half + 2 * ((k & 7) >> 1) * a.chunks + 2 * (k >> 3) + (k & 1) : i;
    turn(turns.t[k], position_of(a, t0 + t), a, cs[at].x, cs[at].y);
  }
  const T *src = static_cast<const T *>(a.src);
  T *dst = static_cast<T *>(a.dst);
  __syncthreads();
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (int(threadIdx.x) + k * kThreads < all) ahead[k].turn_and_store();
    for (int i = threadIdx.x + N * kThreads; i < all; i += kThreads) {
      Chunk<T, IL> c;
      c.load(a, cs, t0, i);
      c.turn_and_store();
    }
  } else {
    for (int i = threadIdx.x; i < all; i += kThreads) {
      const int t = gtp::fast_div(i, a.by_units), r = i - t * a.units;
      const int h = gtp::fast_div(r, a.by_chunks), c = r - h * a.chunks;
      const Head at = head_of(a, t0 + t, h);
      const int ja = IL ? 2 * c : c, jb = IL ? 2 * c + 1 : c + a.half;
      const float x = load_f32(src + at.src + ja), y = load_f32(src + at.src + jb);
      const float2 m = cs[t * a.half + c];
      store_f32(dst + at.dst + ja, x * m.x - y * m.y);
      store_f32(dst + at.dst + jb, x * m.y + y * m.x);
    }
  }
  // the part of a head that keeps its values; in place there is nothing to do
  const int rest = a.head_dim - 2 * a.half;
  if (rest && a.copy) {
    const int per = VEC ? rest / 8 : rest, kept = per * a.heads;
    for (int i = threadIdx.x; i < nt * kept; i += kThreads) {
      const int t = i / kept, r = i - t * kept, h = r / per, c = 2 * a.half + P * (r - h * per);
      const Head at = head_of(a, t0 + t, h);
      if constexpr (VEC) {
        Run<T> u;
        u.load(src + at.src + c);
        u.store(dst + at.dst + c);
      } else {
        dst[at.dst + c] = src[at.src + c];
      }
    }
  }
}

template <typename T, bool VEC>
gtp_status launch(RotaryArgs &a, const Turns &turns, bool interleaved, cudaStream_t st) {
  // As many tokens to a block as fill its threads' chunks, and no more, so that a short batch spreads.  On 8192
  // tokens of 20 heads of 64, 2 / 3 / 4 / 5 / 6 (the rule's) / 8 / 11 / 16: 11.5 / 10.1 / 9.6 / 9.5 / 9.1 / 10.0 /
  // 10.1 / 11.7 us.
  a.chunks = a.half / (VEC ? 8 : 1);
  a.units = a.heads * a.chunks;
  a.by_half = gtp::make_fastdiv(a.half);
  a.by_units = gtp::make_fastdiv(a.units);
  a.by_chunks = gtp::make_fastdiv(a.chunks);
  a.by_group = gtp::make_fastdiv(a.group_heads);
  a.block_tokens =
      int32_t(std::max<int64_t>(1, std::min<int64_t>({Shape<T>::CHUNKS * kThreads / a.units, 16, a.tokens})));
  const unsigned grid = unsigned((a.tokens + a.block_tokens - 1) / a.block_tokens);
  const size_t smem = size_t(a.block_tokens) * a.half * sizeof(float2);
  return interleaved ? gtp::launch_overlapped(rotary_kernel<T, VEC, true>, grid, kThreads, smem, st, "rotary", a, turns)
                     : gtp::launch_overlapped(rotary_kernel<T, VEC, false>, grid, kThreads, smem, st, "rotary", a, turns);
}

template <typename T>
gtp_status launch(RotaryArgs &a, const Turns &turns, bool interleaved, cudaStream_t st) {
  // vectors of 8 elements where every head starts on one (16 bytes, fp32 32) and whole ones turn or stay
  const uintptr_t mask = 8 * sizeof(T) - 1;
  bool vec = !((reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst)) & mask) && a.half % 8 == 0 &&
             a.head_dim % 8 == 0;
  for (int64_t s : {a.src_token, a.src_group, a.src_head, a.dst_token, a.dst_group, a.dst_head})
    vec = vec && s % 8 == 0;
  return vec ? launch<T, true>(a, turns, interleaved, st) : launch<T, false>(a, turns, interleaved, st);
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
  // GTP_ROTARY_RAMP (YaRN, Peng et al. 2023) blends over pair indices, between the (fractional) indices whose
  // frequencies make high_turns and low_turns turns over the context, rounded outwards to whole pairs; the far end is
  // held to rot - 1 and equal ends are set 0.001 apart as its authors released it
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
  if (d->tokens > INT32_MAX || int64_t(d->groups) * d->heads > (1 << 20))
    return gtp::fail(GTP_E_SHAPE, "more than 2^31 - 1 tokens or 2^20 heads");
  // a block walks its tokens' elements in 32 bits
  if (int64_t(d->groups) * d->heads > (int64_t(1) << 30) / d->head_dim)
    return gtp::fail(GTP_E_SHAPE, "more than 2^30 elements in a token's heads");
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
  const gtp::Runs in = {reinterpret_cast<uintptr_t>(d->src), d->head_dim * es,
                        {{d->src_token * es, d->tokens}, {d->src_group * es, d->groups}, {d->src_head * es, d->heads}}};
  const gtp::Runs out = {reinterpret_cast<uintptr_t>(d->dst), d->head_dim * es,
                         {{d->dst_token * es, d->tokens}, {d->dst_group * es, d->groups}, {d->dst_head * es, d->heads}}};
  const bool in_place = d->src == d->dst && (d->tokens == 1 || d->src_token == d->dst_token) &&
                        (d->groups == 1 || d->src_group == d->dst_group) &&
                        (d->heads == 1 || d->src_head == d->dst_head);
  if (!in_place && gtp::overlap(out, in))
    return gtp::fail(GTP_E_ARG, "src and dst overlap and are not the same heads in place");
  if (d->positions && gtp::overlap(gtp::byte_range(d->dst, span * es),
                                    gtp::byte_range(d->positions, d->tokens * (d->positions64 ? 8 : 4))))
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
  a.inverse = d->inverse, a.positions64 = d->positions64, a.copy = !in_place;
  // a stride that no second head uses says nothing about alignment
  if (d->tokens == 1) a.src_token = a.dst_token = 0;
  if (d->groups == 1) a.src_group = a.dst_group = 0;
  if (d->heads == 1) a.src_head = a.dst_head = 0;
  a.scale = d->scale;
  Turns turns = {};
  std::copy(d->turns, d->turns + a.half, turns.t);
  cudaStream_t st = gtp::as_stream(stream);
  return d->dtype == GTP_F32 ? launch<float>(a, turns, d->interleaved, st)
                             : launch<__nv_bfloat16>(a, turns, d->interleaved, st);
}
