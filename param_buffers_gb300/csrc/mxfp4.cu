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

#include "byte_range.h"
#include "device.h"
#include "fastdiv.cuh"
#include "mx4_block.cuh"
#include "philox.cuh"
#include "sm100_ptx.cuh"
#include "wide.cuh"

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
// 32-bit word a row) or of one column twice (fp32), so a column's block needs no shuffle.
//
// Where a word of a tile row lies (in groups of four words, 16 bytes): lanes that store their segments
// are THREAD_WORDS apart, so the low bits of a group are swapped by the bits above them; and the words
// of a row are rotated by 8 per 32 rows, so that the four row blocks of a column, which neighbouring
// lanes hold to write its 64 bytes together, lie in different banks.  Both directions then run without
// bank conflicts.
//
// A source whose rows do not all start on 16 bytes (RAGGED: any odd row length) is read in the 16-byte
// vectors that cover a thread's elements, one more than they fill, and shifted into place in registers.
// Rows 8 apart start at the same place in a vector, so a warp takes such rows and shifts by whole words that are
// known when it is compiled (selecting them by the address took 57 us on [8001, 8191] bf16 against 45).
// Rows' and columns' ends are read past, inside the source, and masked; only the source's own corners, whose
// vectors would reach outside it, go element by element ([1111, 1535]: 7.5 us against 12.4 when every end did).
//
// What bounds it, on [8192, 8192] (share of a copy's rate of the bytes that have to move): to nearest the
// memory, nearly: bf16 both views 35.5 us (86 %), rowwise 26.6 (95 %), columnwise 29.2 (86 %); fp32 55.3 (91 %),
// 44.4 (101 %), 48.0 (94 %).  Stochastically the instructions (74 % of the issue slots, integer and multiply
// pipes 58 %): bf16 both views 55.9 us (54 %), rowwise 33.3, columnwise 34.0; fp32 69.7 (72 %).  Ten rounds of the
// generator, one call for 16 elements of a view, are 17 us of those 55.9 (with two rounds, for the time only,
// 48.0 of 61.9 then), the rounding itself 5.  A ragged source ([8001, 8191] bf16) takes 44.7 us to nearest and
// 61.4 stochastically, fp32 76.6 and 88.3: a third more loads, whose vectors hold the registers.  Blocks that stay
// and copy their next tile into shared memory meanwhile have room for fewer warps: 38.4 and 66.5 us on both bf16 views.
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

// The word of up to two elements, for a ragged or unaligned source.
__device__ __forceinline__ uint32_t word_of(const float *p, int n) { return n > 0 ? __float_as_uint(*p) : 0u; }
__device__ __forceinline__ uint32_t word_of(const __nv_bfloat16 *p, int n) {
  const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
  if (n > 1 && (reinterpret_cast<uintptr_t>(p) & 3u) == 0) return *reinterpret_cast<const uint32_t *>(p);
  return (n > 0 ? uint32_t(q[0]) : 0u) | (n > 1 ? uint32_t(q[1]) << 16 : 0u);
}

struct ViewArgs {
  uint8_t *codes, *scales;
  int64_t pitch;  // bytes of a row of codes
  int64_t words;  // atoms of a 128-row tile
};

struct TileArgs {
  const void *src;
  int64_t rows, cols, ld, src_bytes;
  int64_t tiles_n;
  int32_t wide;  // every row starts on 32 bytes
  ViewArgs row, col;
  gtp::RngArgs rng;
};

// The same in whole sectors.  fp32 takes them where rows allow (both views of [8192, 8192] 66.6 -> 57.7 us);
// bf16, one sector a thread, lost by it (stochastically 60.8 -> 62.0, the rowwise view alone 27.2 -> 28.0).
template <typename T, int N>
__device__ __forceinline__ void load_sectors(const T *p, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    uint32_t v[8];
    gtp::load_32b(p + 8 * Tile<T>::PER * i, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[8 * i + k] = v[k];
  }
}

// The 16-byte vectors around the 16 elements at p, one more than they fill where rows start anywhere, lie inside
// the source.
template <typename T, bool RAGGED>
__device__ __forceinline__ bool window_inside(const T *p, const TileArgs &a) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15), begin = reinterpret_cast<uintptr_t>(a.src);
  return b >= begin && b + 16 * (Tile<T>::THREAD_WORDS / 4 + (RAGGED ? 1 : 0)) <= begin + uintptr_t(a.src_bytes);
}

// 16 elements at an element-aligned address, out of the vectors around them, which start J words and (HALF) one
// bf16 before them.
template <typename T, int J, bool HALF, int N>
__device__ __forceinline__ void load_shifted(const T *p, uint32_t (&w)[N]) {
  constexpr int V = (J + N + (HALF ? 1 : 0) + 3) / 4;  // vectors that hold any of them
  const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
  uint32_t t[4 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint4 v = __ldcs(q + i);
    t[4 * i] = v.x, t[4 * i + 1] = v.y, t[4 * i + 2] = v.z, t[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = HALF ? __funnelshift_r(t[k + J], t[(k + J + 1) % (4 * V)], 16) : t[k + J];
}

// The same of four rows, at these offsets.
template <typename T, int J, int N>
__device__ __forceinline__ void load_rows(const T *p, const int64_t (&off)[4], bool half, uint32_t (&w)[4][N]) {
  if (sizeof(T) == 2 && half) {
#pragma unroll
    for (int it = 0; it < 4; ++it) load_shifted<T, J, sizeof(T) == 2>(p + off[it], w[it]);
  } else {
#pragma unroll
    for (int it = 0; it < 4; ++it) load_shifted<T, J, false>(p + off[it], w[it]);
  }
}

// Index of word `w` of row `r` in the tile.
template <typename T>
__device__ __forceinline__ int word_at(int r, int w) {
  constexpr int WORDS = Tile<T>::WORDS, SPAN = Tile<T>::THREAD_WORDS / 4;
  const int g = w >> 2, s = g ^ ((g >> 3) & (SPAN - 1));
  return r * WORDS + ((4 * s + (w & 3) + 8 * (r >> 5)) & (WORDS - 1));
}

// The largest magnitude of a word's elements so far, as floats (fp32 one, bf16 two); NaN stays.
template <typename T>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t w);
template <>
__device__ __forceinline__ uint32_t max_magnitude<float>(uint32_t m, uint32_t w) {
  float r;
  asm("{\n\t.reg .f32 a;\n\tabs.f32 a, %2;\n\tmax.NaN.f32 %0, %1, a;\n\t}"
      : "=f"(r)
      : "f"(__uint_as_float(m)), "f"(__uint_as_float(w)));
  return __float_as_uint(r);
}
template <>
__device__ __forceinline__ uint32_t max_magnitude<__nv_bfloat16>(uint32_t m, uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  return r;
}

__device__ __forceinline__ float low_f32(uint32_t w) { return __uint_as_float(w << 16); }

// Two values in a pair, divided by the block's scale.  bf16 elements, the low or the high halves of two words, are
// multiplied as they lie by a product of halves added to -0, which keeps the sign of zero: half of the unpacking
// gone (both views of [8192, 8192] bf16 36.7 -> 36.2 us, stochastically 60.1 -> 57.7).
__device__ __forceinline__ uint64_t scaled(float a, float b, float inv) {
  return gtp::mx4::mul2(gtp::mx4::pack2(a, b), gtp::mx4::pack2(inv, inv));
}
__device__ __forceinline__ float scaled_half(uint32_t w, bool high, float inv) {
  float r;
  if (high)
    asm("{\n\t.reg .b16 l, h, z, s;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {z, s}, %2;\n\t"
        "fma.rn.f32.bf16 %0, h, s, %3;\n\t}"
        : "=f"(r)
        : "r"(w), "f"(inv), "f"(-0.f));
  else
    asm("{\n\t.reg .b16 l, h, z, s;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {z, s}, %2;\n\t"
        "fma.rn.f32.bf16 %0, l, s, %3;\n\t}"
        : "=f"(r)
        : "r"(w), "f"(inv), "f"(-0.f));
  return r;
}
__device__ __forceinline__ uint64_t scaled_halves(uint32_t a, bool a_high, uint32_t b, bool b_high, float inv) {
  return gtp::mx4::pack2(scaled_half(a, a_high, inv), scaled_half(b, b_high, inv));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Far blocks' values brought near (mx4::near_factor; one product an element fewer for all the others, both views of
// [8192, 8192] bf16 57.4 -> 55.9 us), on the words as they lie, so that the branch, which
// real data hardly takes, holds no registers of its own: one block's, or (bf16) those of the low and the high halves.
template <typename T, int N>
__device__ __forceinline__ void bring_near(uint32_t (&w)[N], uint32_t low, uint32_t high) {
  if (!(gtp::mx4::is_far(low) || gtp::mx4::is_far(high))) return;
  const uint32_t f0 = __float_as_uint(gtp::mx4::near_factor(low)), f1 = __float_as_uint(gtp::mx4::near_factor(high));
#pragma unroll
  for (int i = 0; i < N; ++i)
    w[i] = sizeof(T) == 2 ? mul_bf16x2(w[i], f0 >> 16 | (f1 & 0xFFFF0000u))
                          : __float_as_uint(__uint_as_float(w[i]) * __uint_as_float(f0));
}

// 2 N values in pairs, divided by the scale of their block's `byte`, to codes; view row r and its first group of draws.
template <bool STOCH, int N>
__device__ __forceinline__ void encode_run(const uint64_t (&x)[N], uint32_t byte, uint32_t (&w)[N / 4], uint32_t stream,
                                           uint32_t r, uint32_t first_group, const gtp::RngArgs &rng, uint64_t offset) {
#pragma unroll
  for (int h = 0; h < N / 8; ++h) {
    uint4 d = make_uint4(0, 0, 0, 0);
    if (STOCH)
      d = gtp::philox(rng, (first_group + h) | (stream << 30), r, uint32_t(offset), uint32_t(offset >> 32));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint64_t v[4] = {x[8 * h + 4 * q], x[8 * h + 4 * q + 1], x[8 * h + 4 * q + 2], x[8 * h + 4 * q + 3]};
      w[2 * h + q] = STOCH ? gtp::mx4::codes8_stochastic(v, q ? d.z : d.x, q ? d.w : d.y) : gtp::mx4::codes8(v);
    }
  }
  if (byte == gtp::mx4::kNanScale) {  // a bad block's codes are 0
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = 0;
  }
}

// Blocks an SM that the registers are held to: latency against spills.  On [8192, 8192], 2 / 3 / 4 blocks: bf16
// both views 45.8 / 39.4 / 37.2 us to nearest and 67.8 / 62.0 / 61.8 stochastically; fp32 both views 57.6 / 66.6 /
// 92.2 (its 64 registers of tile words spill from 3 on), but the rowwise view alone 46.7 / 44.6 / 48.8 (all before
// the maxima and the scaling took fewer instructions).  A ragged fp32 rowwise view 49.7 with 2, 67.6 with 3.
template <typename T, bool COL, bool RAGGED>
constexpr int kMinBlocks = sizeof(T) == 2 ? 4 : COL || RAGGED ? 2 : 3;

template <typename T, bool STOCH, bool ROW, bool COL, bool RAGGED>
__global__ void __launch_bounds__(kThreads, kMinBlocks<T, COL, RAGGED>)
    mx4_tile_kernel(const __grid_constant__ TileArgs a) {
  using F = Tile<T>;
  constexpr int TW = F::THREAD_WORDS;
  extern __shared__ __align__(16) uint32_t tile[];  // COL: [128][WORDS]
  __shared__ __align__(16) uint8_t atom[2][512];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const uint64_t offset = STOCH ? gtp::rng_offset(a.rng) : 0;
  const int tid = threadIdx.x;
  const int64_t tm = blockIdx.x / a.tiles_n, tn = blockIdx.x - tm * a.tiles_n;
  // this thread's 16 columns, and its row of every 32; a warp's rows are 8 apart where rows start anywhere, so that
  // they all start at the same place in a vector
  const int seg = tid & 7, r32 = RAGGED ? (tid >> 5) + 8 * ((tid >> 3) & 3) : tid >> 3;
  const int64_t c0 = kTile * tn + 16 * seg;
  const int nc = int(max(int64_t(0), min(int64_t(16), a.cols - c0)));  // its columns inside the matrix
  uint32_t w[4][TW];
  const int64_t r0 = kTile * tm + r32;
  const int nr = int(max(int64_t(0), min(int64_t(4), (a.rows - r0 + 31) >> 5)));  // its rows inside
  const T *p = static_cast<const T *>(a.src) + r0 * a.ld + c0;
  const auto load = [&](const T *q, uint32_t(&v)[TW]) {
    if (sizeof(T) == 4 && a.wide)
      load_sectors(q, v);
    else
      load_words(reinterpret_cast<const uint32_t *>(q), v);
  };
  if (!RAGGED && nr == 4 && nc == 16) {
#pragma unroll
    for (int it = 0; it < 4; ++it) load(p + 32 * it * a.ld, w[it]);
  } else if (nr == 0 || nc == 0) {
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int i = 0; i < TW; ++i) w[it][i] = 0;
  } else {
    int64_t off[4];  // rows past the end read the first one again
#pragma unroll
    for (int it = 0; it < 4; ++it) off[it] = it < nr ? 32 * it * a.ld : 0;
    // vectors where they lie inside the source, even past a row's end; the elements one by one at its corners
    if (window_inside<T, RAGGED>(p, a) && window_inside<T, RAGGED>(p + 32 * (nr - 1) * a.ld, a)) {
      if constexpr (RAGGED) {
        const uint32_t s = uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;
        const bool half = (s & 2u) != 0;
        if (s < 4)
          load_rows<T, 0>(p, off, half, w);
        else if (s < 8)
          load_rows<T, 1>(p, off, half, w);
        else if (s < 12)
          load_rows<T, 2>(p, off, half, w);
        else
          load_rows<T, 3>(p, off, half, w);
      } else {
#pragma unroll
        for (int it = 0; it < 4; ++it) load(p + off[it], w[it]);
      }
    } else {
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int i = 0; i < TW; ++i) w[it][i] = word_of(p + off[it] + F::PER * i, nc - F::PER * i);
    }
    if (nr < 4 || nc < 16) {
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int i = 0; i < TW; ++i) {
          const int n = it < nr ? nc - F::PER * i : 0;  // elements of the word inside
          w[it][i] = n >= F::PER ? w[it][i] : n > 0 ? w[it][i] & 0xFFFFu : 0u;
        }
    }
  }
  if (COL) {
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int i = 0; i < TW / 4; ++i)
        *reinterpret_cast<uint4 *>(tile + word_at<T>(32 * it + r32, seg * TW + 4 * i)) =
            make_uint4(w[it][4 * i], w[it][4 * i + 1], w[it][4 * i + 2], w[it][4 * i + 3]);
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
      const float inv = STOCH ? gtp::mx4::down_factor(byte) : gtp::mx4::inv_scale(byte);
      if (STOCH) bring_near<T>(w[it], byte, byte);
      uint64_t x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = sizeof(T) == 4
                   ? scaled(__uint_as_float(w[it][2 * k % TW]), __uint_as_float(w[it][(2 * k + 1) % TW]), inv)
                   : scaled_halves(w[it][k % TW], false, w[it][k % TW], true, inv);
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
      const uint32_t *t = tile + word_at<T>(32 * rb, p);  // the rows of a block share the word's place
      uint32_t v[32], m = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        v[k] = t[k * F::WORDS];
        m = max_magnitude<T>(m, v[k]);
      }
      const uint32_t b0 = gtp::mx4::scale_byte<STOCH>(F::PER == 1 ? m : m << 16);
      const uint32_t b1 = gtp::mx4::scale_byte<STOCH>(F::PER == 1 ? m : m & 0xFFFF0000u);
      if (STOCH) bring_near<T>(v, b0, b1);
#pragma unroll
      for (int e = 0; e < F::PER; ++e) {
        const int c = F::PER * p + e;
        const int64_t gc = kTile * tn + c;
        const uint32_t byte = e ? b1 : b0;
        const float inv = STOCH ? gtp::mx4::down_factor(byte) : gtp::mx4::inv_scale(byte);
        uint64_t x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          x[k] = F::PER == 1 ? scaled(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]), inv)
                             : scaled_halves(v[2 * k], e, v[2 * k + 1], e, inv);
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
    reinterpret_cast<uint4 *>(a.row.scales + (tm * a.row.words + tn) * 512)[tid] =
        reinterpret_cast<uint4 *>(atom[0])[tid];
  if (COL && tid >= 32 && tid < 64)
    reinterpret_cast<uint4 *>(a.col.scales + (tn * a.col.words + tm) * 512)[tid - 32] =
        reinterpret_cast<uint4 *>(atom[1])[tid - 32];
}

// Values back from a view, exact in bf16 and fp32 below 2^128 (one mantissa bit; the smallest
// magnitude, 2^-128, is a bf16 subnormal).  A code's bf16 magnitude comes from a table of 8 in two
// byte permutes for four codes, its sign by a multiply that moves two sign bits at once, and the scale
// by a bf16 product, exact because it is a power of two.
//
// A thread writes sixteen elements, half a block, where they lie on whole 32-byte sectors of the output.
// Where rows start anywhere (SHIFTED: an odd length), those are the elements from `head` + 16 v on, head
// the row's elements before its first such place: out of its own two words and those of the lane above
// (the last lane of a warp only reads), under up to two scale bytes.  Items (row, v) run over all rows'
// half blocks, narrow rows side by side in a warp; the up to 15 elements at either end of a shifted row
// go one by one, a thread each, in the blocks after the others.
//
// The bytes bound it: [8192, 8192] bf16 26.2 us (96 % of a copy's rate), fp32 45.0 (100 %); [8192, 8001] bf16,
// shifted, 34.2 (72 %: the integer work of the shifts).
__device__ __forceinline__ uint32_t scale_bf16(uint32_t byte) {
  return byte == gtp::mx4::kNanScale ? 0x7FC0u : byte == 0 ? 0x0040u : byte << 7;
}

// Two codes in the low byte of w to two bf16 values; mag: their magnitudes.
__device__ __forceinline__ uint32_t with_signs(uint32_t mag, uint32_t w) {
  return mag | (((w & 0x88u) * 0x1001000u) & 0x80008000u);  // bits 3 and 7 to 15 and 31
}

struct ValueArgs {
  const uint8_t *codes, *scales;
  void *out;
  int64_t rows, len, blocks, words;
  int64_t row0;           // rows before these in the view (a later launch of one call)
  int32_t items, groups;  // half blocks of all rows and of a row that hold elements
  int32_t vector_blocks;
  gtp::FastDiv by_groups;
};

__device__ __forceinline__ uint32_t scale_byte_at(const ValueArgs &a, int64_t row, int64_t b) {
  const int64_t r = row + a.row0;
  return a.scales[((r >> 7) * a.words + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3)];
}

constexpr int kValueItems = 2;  // items a thread has in flight

template <typename T, bool SHIFTED>
__global__ void __launch_bounds__(kThreads) mx4_values_kernel(const __grid_constant__ ValueArgs a) {
  constexpr int N = kValueItems, PER = SHIFTED ? 31 : 32;
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  T *out = static_cast<T *>(a.out);
  const auto head_of = [&](int64_t row) {
    return int((0u - uint32_t(reinterpret_cast<uintptr_t>(out + row * a.len) / sizeof(T))) & 15u);
  };
  if (SHIFTED && int(blockIdx.x) >= a.vector_blocks) {  // the ends: 32 threads a row
    const int64_t i = int64_t(blockIdx.x - a.vector_blocks) * kThreads + threadIdx.x, row = i >> 5;
    if (row >= a.rows) return;
    const int e = int(i & 31);
    const int64_t head = min(int64_t(head_of(row)), a.len), tail = head + (a.len - head) / 16 * 16;
    const int64_t j = e < 16 ? e : tail + e - 16;
    if (e < 16 ? j >= head : j >= a.len) return;
    const uint32_t c = uint32_t(a.codes[row * a.blocks * 16 + (j >> 1)]) >> (4 * (j & 1)), m = c & 7u;
    const uint32_t mag = (__byte_perm(0xC0800000u, 0xC0804000u, m) & 0xFFu) |
                         (__byte_perm(0x3F3F3F00u, 0x40404040u, m) & 0xFFu) << 8;
    const uint32_t v = mul_bf16x2(mag | (c & 8u) << 12, scale_bf16(scale_byte_at(a, row, j >> 5)));
    out[row * a.len + j] = T(low_f32(v));
    return;
  }
  const int lane = threadIdx.x & 31;
  const int first = (int(blockIdx.x) * (kThreads / 32) + int(threadIdx.x >> 5)) * N * PER + lane;
  uint2 w[N];
  uint32_t s[N];
  int row[N], g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int item = min(first + i * PER, a.items - 1);
    row[i] = gtp::fast_div(item, a.by_groups);
    g[i] = item - row[i] * a.groups;
    w[i] = __ldcs(reinterpret_cast<const uint2 *>(a.codes + int64_t(row[i]) * a.blocks * 16) + g[i]);
    s[i] = scale_byte_at(a, row[i], g[i] >> 1);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t c[2] = {w[i].x, w[i].y}, ab = scale_bf16(s[i]);
    int head = 0;
    if (SHIFTED) {
      // where head > 0 the vector reaches into half block g + 1 of the same row, which exists
      head = head_of(row[i]);
      const uint32_t n0 = __shfl_down_sync(0xFFFFFFFFu, c[0], 1), n1 = __shfl_down_sync(0xFFFFFFFFu, c[1], 1);
      ab |= __shfl_down_sync(0xFFFFFFFFu, ab, 1) << 16;
      const bool far = head >= 8;
      const uint32_t x = far ? c[1] : c[0], y = far ? n0 : c[1], z = far ? n1 : n0;
      c[0] = __funnelshift_r(x, y, 4 * (head & 7));
      c[1] = __funnelshift_r(y, z, 4 * (head & 7));
    }
    const int64_t j = int64_t(head) + 16 * int64_t(g[i]);
    if (first + i * PER >= a.items || (SHIFTED && (lane == 31 || j + 16 > a.len))) continue;
    uint32_t v[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // four codes a round
      const uint32_t q = c[h >> 1] >> (16 * (h & 1)), sel = q & 0x7777u;
      const uint32_t top = __byte_perm(0x3F3F3F00u, 0x40404040u, sel), low = __byte_perm(0xC0800000u, 0xC0804000u, sel);
      v[2 * h] = with_signs(__byte_perm(low, top, 0x5140), q);
      v[2 * h + 1] = with_signs(__byte_perm(low, top, 0x7362), q >> 8);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {  // elements from 16 - head on are the next half block's
      const uint32_t sel = !SHIFTED || 2 * p + 1 < 16 - head ? 0x1010u : 2 * p < 16 - head ? 0x3210u : 0x3232u;
      v[p] = mul_bf16x2(v[p], __byte_perm(ab, 0, sel));
    }
    T *o = out + int64_t(row[i]) * a.len + j;
    if constexpr (sizeof(T) == 2) {
      gtp::store_32b(o, v);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) f[2 * p] = v[4 * h + p] << 16, f[2 * p + 1] = v[4 * h + p] & 0xFFFF0000u;
        gtp::store_32b(o + 8 * h, f);
      }
    }
  }
}

template <typename T>
gtp_status launch_values(ValueArgs a, cudaStream_t st) {
  const bool shifted = reinterpret_cast<uintptr_t>(a.out) % (16 * sizeof(T)) || a.len % 16 != 0;
  a.groups = int32_t((a.len + 15) / 16);
  a.by_groups = gtp::make_fastdiv(a.groups);
  // items are counted in 31 bits: more than 2^30 half blocks go in several launches
  const int64_t rows = a.rows, most = std::max<int64_t>(1, (int64_t(1) << 30) / a.groups);
  const uint8_t *codes = a.codes;
  T *out = static_cast<T *>(a.out);
  for (int64_t r = 0; r < rows; r += most) {
    a.row0 = r;
    a.rows = std::min(most, rows - r);
    a.codes = codes + r * a.blocks * 16;
    a.out = out + r * a.len;
    a.items = int32_t(a.rows * a.groups);
    const int64_t a_block = (kThreads / 32) * kValueItems * (shifted ? 31 : 32);
    a.vector_blocks = int32_t((a.items + a_block - 1) / a_block);
    const int64_t ends = shifted ? (a.rows * 32 + kThreads - 1) / kThreads : 0;
    const unsigned grid = unsigned(a.vector_blocks + ends);
    const gtp_status e =
        shifted ? gtp::launch_overlapped(mx4_values_kernel<T, true>, grid, kThreads, 0, st, "mxfp4_dequantize", a)
                : gtp::launch_overlapped(mx4_values_kernel<T, false>, grid, kThreads, 0, st, "mxfp4_dequantize", a);
    if (e) return e;
  }
  return GTP_OK;
}

struct View {
  uint8_t *codes, *scales;
  int64_t rows, len;
  int64_t blocks() const { return (len + 31) / 32; }
  int64_t words() const { return (blocks() + 3) / 4; }
  int64_t code_bytes() const { return rows * blocks() * 16; }
  int64_t scale_bytes() const { return (rows + 127) / 128 * words() * 512; }
};

template <typename T, bool STOCH, bool ROW, bool COL, bool RAGGED>
gtp_status launch_tiles(const TileArgs &a, int64_t tiles, const gtp::DeviceInfo &dev, cudaStream_t st) {
  constexpr int smem = COL ? Tile<T>::BYTES : 0;
  constexpr auto kernel = mx4_tile_kernel<T, STOCH, ROW, COL, RAGGED>;
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

template <typename T, bool STOCH, bool RAGGED>
gtp_status launch_views(const TileArgs &a, int64_t tiles, const gtp::DeviceInfo &dev, cudaStream_t st) {
  if (!a.col.codes) return launch_tiles<T, STOCH, true, false, RAGGED>(a, tiles, dev, st);
  if (!a.row.codes) return launch_tiles<T, STOCH, false, true, RAGGED>(a, tiles, dev, st);
  return launch_tiles<T, STOCH, true, true, RAGGED>(a, tiles, dev, st);
}

template <typename T>
gtp_status launch_views(const TileArgs &a, bool stochastic, int64_t tiles, const gtp::DeviceInfo &dev,
                        cudaStream_t st) {
  const bool ragged = !gtp::aligned16(a.src) || a.ld * int64_t(sizeof(T)) % 16 != 0;
  if (stochastic)
    return ragged ? launch_views<T, true, true>(a, tiles, dev, st) : launch_views<T, true, false>(a, tiles, dev, st);
  return ragged ? launch_views<T, false, true>(a, tiles, dev, st) : launch_views<T, false, false>(a, tiles, dev, st);
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
  if (rows > 1 && src_ld > (int64_t(1) << 50) / rows) return gtp::fail(GTP_E_SHAPE, "src spans more than 2^50 elements");
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
  a.src_bytes = ((rows - 1) * a.ld + cols) * es;
  a.tiles_n = (cols + kTile - 1) / kTile;
  a.row = {row_codes, row_scales, row.blocks() * 16, row.words()};
  a.col = {col_codes, col_scales, col.blocks() * 16, col.words()};
  a.wide = ((reinterpret_cast<uintptr_t>(src) | uintptr_t(a.ld * es)) & 31u) == 0;
  a.rng = gtp::rng_args(rng);
  const int64_t tiles = (rows + kTile - 1) / kTile * a.tiles_n;
  if (tiles > INT32_MAX) return gtp::fail(GTP_E_SHAPE, "more than 2^31 - 1 tiles of 128 x 128");
  return src_dt == GTP_F32 ? launch_views<float>(a, rng != nullptr, tiles, dev, st)
                           : launch_views<__nv_bfloat16>(a, rng != nullptr, tiles, dev, st);
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
  ValueArgs a = {};
  a.codes = codes, a.scales = scales, a.out = out;
  a.rows = rows, a.len = cols, a.blocks = v.blocks(), a.words = v.words();
  return out_dt == GTP_F32 ? launch_values<float>(a, st) : launch_values<__nv_bfloat16>(a, st);
}
