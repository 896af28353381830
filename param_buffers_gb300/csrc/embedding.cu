// Token embedding of a vocabulary shard, and its gradient accumulated into the flat gradient buffer by sorted tokens.
//
// Pages: "Megatron-LM architecture and source guide" (arganzheng.life), §1 (the embedding before the first layer) and
// "05 · grad/param buffer ..." (llm-infra-atlas), §4.2 and §5 (the embedding's bucket, main_grad as a view).
//
//   out[t] = scale * table[ids[t] - first_row]  where that row is in the shard, else 0
//   grad[r] += scale * sum of dout[t] over the tokens t of row r
// The gradient's sum over a row's tokens is formed in fp32 in an order that depends on the ids alone: tokens are sorted
// by row (ties in token order), the sorted list is cut into tiles of equal length, a row inside a tile is summed and
// added at once, a row that crosses tiles leaves one part a tile, and whoever leaves the last part adds them all up in
// their order.  No atomic's order takes part, so equal calls give equal bits.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "byte_range.h"
#include "device.h"
#include "eight.cuh"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kThreads = 256;

// As two 32-bit words (one of them twice where the ids are 32 bits wide): without a branch several ids' loads are under
// way at once.
__device__ __forceinline__ int64_t id_at(const void *ids, int wide, int64_t t) {
  const int32_t *const p = static_cast<const int32_t *>(ids) + (t << wide);
  const int32_t low = p[0], high = p[wide];
  return wide ? int64_t(uint64_t(uint32_t(high)) << 32 | uint32_t(low)) : int64_t(low);
}

// The shard's row of a token, or `rows` for one of another shard (or of none).  Unsigned: no id wraps into the range.
__device__ __forceinline__ int64_t row_of(const void *ids, int wide, int64_t t, int64_t first_row, int64_t rows) {
  const uint64_t r = uint64_t(id_at(ids, wide, t)) - uint64_t(first_row);
  return r < uint64_t(rows) ? int64_t(r) : rows;
}

// Eight elements of a row that one thread moves: consecutive ones (VEC), as they lie in memory, or every
// step-th from its own on, so that a warp's accesses stand side by side whatever the row's alignment; n of them exist.
template <typename T, bool VEC>
struct Group {
  gtp::Eight<T> e;
  __device__ __forceinline__ void load(const T *p, int, int) { e.load(p); }
  __device__ __forceinline__ void clear() { e.clear(); }
  __device__ __forceinline__ void get(float (&x)[8]) const { e.get(x); }
  static __device__ __forceinline__ void store(T *p, int, int, const float (&x)[8]) {
    gtp::Eight<T> v;
    v.set(x);
    v.store(p);
  }
};
template <typename T>
struct Group<T, false> {
  T v[8];
  __device__ __forceinline__ void load(const T *p, int step, int n) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k * step] : T(0.f);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = T(0.f);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = float(v[k]);
  }
  static __device__ __forceinline__ void store(T *p, int step, int n, const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k * step] = T(x[k]);
  }
};

// A block is tx threads wide, eight columns a thread; this thread's first column and how many of its eight exist.
template <bool VEC>
__device__ __forceinline__ bool columns(int64_t cols, int64_t &c, int &n) {
  const int tx = blockDim.x;
  const int64_t c0 = int64_t(blockIdx.x) * 8 * tx;
  c = c0 + (VEC ? 8 * threadIdx.x : threadIdx.x);
  if (c >= cols) return false;
  n = VEC ? 8 : int(min(int64_t(8), (cols - c + tx - 1) / tx));
  return true;
}

// --------------------------------------------------------------------------- lookup

struct LookupArgs {
  const void *ids, *table;
  void *out;
  int64_t tokens, table_ld, out_ld, first_row, rows, cols;
  float scale;
  int wide;
};

// N tokens of a thread in flight: their ids, then their rows.
template <typename TI, typename TO, bool VEC, int N>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const __grid_constant__ LookupArgs a) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  int64_t c;
  int n;
  if (!columns<VEC>(a.cols, c, n)) return;
  const int tx = blockDim.x;
  const int64_t step = int64_t(gridDim.y) * blockDim.y;
  for (int64_t t0 = int64_t(blockIdx.y) * blockDim.y + threadIdx.y; t0 < a.tokens; t0 += N * step) {
    int64_t row[N];
    Group<TI, VEC> x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t t = t0 + i * step;
      row[i] = t < a.tokens ? row_of(a.ids, a.wide, t, a.first_row, a.rows) : a.rows;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i].clear();
      if (row[i] < a.rows) x[i].load(static_cast<const TI *>(a.table) + row[i] * a.table_ld + c, tx, n);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t t = t0 + i * step;
      if (t >= a.tokens) continue;
      float y[8];
      x[i].get(y);
      if (row[i] < a.rows) {  // not the zeros of other shards' tokens: a scale of Inf or NaN leaves them 0
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] *= a.scale;
      }
      Group<TO, VEC>::store(static_cast<TO *>(a.out) + t * a.out_ld + c, tx, n, y);
    }
  }
}

// --------------------------------------------------------------------------- sorting the tokens

// Sorted lists: key[p] the row, token[p] the token of sorted place p; places behind the shard's tokens hold key `rows`.
struct SortArgs {
  const void *ids;
  int64_t first_row, rows;
  int32_t tokens, wide;
  int32_t *key, *token;  // the result
  int32_t *key2, *token2;
  int32_t *counts;  // radix: [256][tiles], or without scan [tiles][256]
  int32_t tiles, scan;
  int32_t *counters;  // of the sums, cleared here
  int64_t counter_count;
};

__device__ __forceinline__ void clear_counters(const SortArgs &a) {
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < a.counter_count; i += int64_t(gridDim.x) * blockDim.x)
    a.counters[i] = 0;
}

// Few tokens: the place of a token is the number of tokens that sort before it, counted outright.  A block owns
// kOwn tokens, keeps every token of the shard as one 32-bit number row * tokens + t in shared memory (any order: the
// numbers differ), and its warps count, 32 owned tokens a warp, each over a part of the list.  tokens^2 comparisons
// but one launch and no exchange between blocks: the whole gradient of [2048, 256] takes 15.0 us, 16.4 with the radix
// sort; at 4096 tokens 21.5 and 19.6.
constexpr int kOwn = 64, kRankThreads = 512, kRankMost = 2560;

__global__ void __launch_bounds__(kRankThreads) rank_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ __align__(16) uint32_t list[];  // tokens rounded up to 4, padded with the largest number
  __shared__ uint32_t own[kOwn], place[kOwn];
  __shared__ int listed, owned;
  gtp::ptx::allow_dependents();
  if (threadIdx.x == 0) listed = owned = 0;
  if (threadIdx.x < kOwn) place[threadIdx.x] = 0;
  gtp::ptx::wait_prior_grid();
  clear_counters(a);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = blockIdx.x * kOwn;
  constexpr int N = 8;  // ids of a thread in flight
  for (int t0 = 32 * warp; t0 < a.tokens; t0 += N * kRankThreads) {
    int64_t row[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = t0 + i * kRankThreads + lane;
      row[i] = t < a.tokens ? row_of(a.ids, a.wide, t, a.first_row, a.rows) : a.rows;
    }
    unsigned m[N];
    int total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m[i] = __ballot_sync(0xFFFFFFFFu, row[i] < a.rows);
      total += __popc(m[i]);
    }
    int base = 0;
    if (lane == 0 && total) base = atomicAdd(&listed, total);
    base = __shfl_sync(0xFFFFFFFFu, base, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = t0 + i * kRankThreads + lane;
      if (row[i] < a.rows) {
        const uint32_t k = uint32_t(row[i]) * uint32_t(a.tokens) + uint32_t(t);
        list[base + __popc(m[i] & ((1u << lane) - 1))] = k;
        if (t >= first && t < first + kOwn) own[atomicAdd(&owned, 1)] = k;
      }
      base += __popc(m[i]);
    }
  }
  __syncthreads();
  const int n = listed, mine = owned;
  if (threadIdx.x < 4 && n + threadIdx.x < ((n + 3) & ~3)) list[n + threadIdx.x] = 0xFFFFFFFFu;
  __syncthreads();
  const int sets = (mine + 31) >> 5;  // of 32 owned tokens
  if (sets > 0) {
    const int parts = (kRankThreads / 32) / sets, set = warp % sets, part = warp / sets;
    if (part < parts) {
      const int i = 32 * set + lane;
      const uint32_t k = i < mine ? own[i] : 0u;
      const int quads = (n + 3) >> 2, q0 = int(int64_t(quads) * part / parts), q1 = int(int64_t(quads) * (part + 1) / parts);
      uint32_t before = 0;
#pragma unroll 4
      for (int q = q0; q < q1; ++q) {
        const uint4 v = reinterpret_cast<const uint4 *>(list)[q];
        before += (v.x < k) + (v.y < k) + (v.z < k) + (v.w < k);
      }
      if (i < mine) atomicAdd(&place[i], before);
    }
  }
  __syncthreads();
  if (threadIdx.x < mine) {
    const uint32_t k = own[threadIdx.x], p = place[threadIdx.x];
    a.key[p] = int32_t(k / uint32_t(a.tokens));
    a.token[p] = int32_t(k % uint32_t(a.tokens));
  }
  if (threadIdx.x < kOwn) {  // the places behind the shard's tokens
    const int p = first + int(threadIdx.x);
    if (p >= n && p < a.tokens) a.key[p] = int32_t(a.rows);
  }
}

// Many tokens: a radix sort from the low digit up, eight bits a pass: digits counted by tiles of 512 tokens (2048 of many),
// the counts summed up in (digit, tile) order, and each tile's tokens written to their places in order.  The first pass
// reads the ids themselves.
constexpr int kTileThreads = 256;

__device__ __forceinline__ void radix_load(const SortArgs &a, const int32_t *key, const int32_t *token, int64_t p,
                                           int32_t &k, int32_t &t) {
  if (key) {
    k = key[p];
    t = token[p];
  } else {
    k = int32_t(row_of(a.ids, a.wide, p, a.first_row, a.rows));
    t = int32_t(p);
  }
}

template <int ROUNDS>
__global__ void __launch_bounds__(kTileThreads)
    radix_count_kernel(const __grid_constant__ SortArgs a, const int32_t *key, int shift) {
  __shared__ int32_t count[256];
  gtp::ptx::allow_dependents();
  count[threadIdx.x] = 0;
  gtp::ptx::wait_prior_grid();
  if (shift == 0) clear_counters(a);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int64_t p = (int64_t(blockIdx.x) * ROUNDS + i) * kTileThreads + threadIdx.x;
    if (p < a.tokens) {
      const int32_t k = key ? key[p] : int32_t(row_of(a.ids, a.wide, p, a.first_row, a.rows));
      atomicAdd(&count[(k >> shift) & 255], 1);
    }
  }
  __syncthreads();
  a.counts[a.scan ? int64_t(threadIdx.x) * a.tiles + blockIdx.x : blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

// counts -> what stands before each, in place, by one block.
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) radix_scan_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int32_t sums[32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = int64_t(256) * a.tiles;
  int32_t carry = 0;
  for (int64_t i0 = 0; i0 < n; i0 += 4 * kScanThreads) {
    int32_t v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + 4 * threadIdx.x + k;
      v[k] = i < n ? a.counts[i] : 0;
      sum += v[k];
    }
    int32_t run = sum;  // inclusive over the warp
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int32_t o = __shfl_up_sync(0xFFFFFFFFu, run, d);
      if (lane >= d) run += o;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    if (warp == 0) {
      int32_t s = sums[lane];
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += o;
      }
      sums[lane] = s;
    }
    __syncthreads();
    int32_t before = carry + (warp ? sums[warp - 1] : 0) + run - sum;
    carry += sums[31];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + 4 * threadIdx.x + k;
      if (i < n) a.counts[i] = before;
      before += v[k];
    }
  }
}

// Up to kFewTiles each block adds up the counts itself (not SCANNED): a launch less.
constexpr int kFewTiles = 64;

// Thread d: the tokens that stand before the tile's first one of digit d.  sums: 8 words.
__device__ __forceinline__ int32_t before_digit(const SortArgs &a, int32_t *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t total = 0, mine = 0;
  for (int i0 = 0; i0 < a.tiles; i0 += 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int32_t c = i0 + i < a.tiles ? a.counts[(i0 + i) * 256 + threadIdx.x] : 0;
      total += c;
      mine += i0 + i < int(blockIdx.x) ? c : 0;
    }
  }
  int32_t run = total;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int32_t o = __shfl_up_sync(0xFFFFFFFFu, run, d);
    if (lane >= d) run += o;
  }
  if (lane == 31) sums[warp] = run;
  __syncthreads();
  for (int w = 0; w < warp; ++w) run += sums[w];
  return run - total + mine;
}

template <int ROUNDS, bool SCANNED>
__global__ void __launch_bounds__(kTileThreads)
    radix_scatter_kernel(const __grid_constant__ SortArgs a, const int32_t *key, const int32_t *token, int32_t *key_out,
                         int32_t *token_out, int shift) {
  __shared__ int32_t at[kTileThreads / 32][256];  // a warp's next place of each digit
  __shared__ int32_t sums[kTileThreads / 32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = 0; w < kTileThreads / 32; ++w) at[w][threadIdx.x] = 0;
  __syncthreads();
  // a warp takes an eighth of the tile's tokens in a row, 32 at a time
  const int64_t p0 = (int64_t(blockIdx.x) * kTileThreads + warp * 32) * ROUNDS + lane;
  int32_t k[ROUNDS], t[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int64_t p = p0 + 32 * i;
    k[i] = t[i] = 0;
    if (p < a.tokens) {
      radix_load(a, key, token, p, k[i], t[i]);
      atomicAdd(&at[warp][(k[i] >> shift) & 255], 1);
    }
  }
  __syncthreads();
  {  // thread d: digit d's place for each warp in turn
    int32_t before = SCANNED ? a.counts[int64_t(threadIdx.x) * a.tiles + blockIdx.x] : before_digit(a, sums);
    for (int w = 0; w < kTileThreads / 32; ++w) {
      const int32_t c = at[w][threadIdx.x];
      at[w][threadIdx.x] = before;
      before += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const bool live = p0 + 32 * i < a.tokens;
    const int d = live ? (k[i] >> shift) & 255 : 256 + lane;  // no one's digit
    const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
    const int rank = __popc(same & ((1u << lane) - 1));
    int32_t base = 0;
    if (live) base = at[warp][d];
    __syncwarp();
    if (live && rank == 0) at[warp][d] = base + __popc(same);
    __syncwarp();
    if (live) {
      key_out[base + rank] = k[i];
      token_out[base + rank] = t[i];
    }
  }
}

// --------------------------------------------------------------------------- the rows' sums

struct SumArgs {
  const int32_t *key, *token;
  const void *dout;
  void *grad;
  float *part;  // [tiles][2][cols]: the row that comes in from the tile before, and the one that goes on
  int32_t *counters;  // [tiles][3][groups]
  int64_t dout_ld, rows, cols;
  int32_t tokens, tile, tiles, groups;  // groups: warps across a row
  float scale;
};

// grad[row] += scale * x at this thread's eight columns: one rounding of the sum in the buffer's type.  fp32 by the
// memory's own additions: nobody else adds to these elements in this call, so the result does not depend on their order.
template <bool VEC>
__device__ __forceinline__ void add8(float *p, int step, int n, float scale, const float (&x)[8]) {
  if (VEC) {
    atomicAdd(reinterpret_cast<float4 *>(p), make_float4(scale * x[0], scale * x[1], scale * x[2], scale * x[3]));
    atomicAdd(reinterpret_cast<float4 *>(p) + 1, make_float4(scale * x[4], scale * x[5], scale * x[6], scale * x[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) atomicAdd(p + k * step, scale * x[k]);
  }
}
template <bool VEC>
__device__ __forceinline__ void add8(__nv_bfloat16 *p, int step, int n, float scale, const float (&x)[8]) {
  Group<__nv_bfloat16, VEC> v;
  v.load(p, step, n);
  float g[8];
  v.get(g);
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = fmaf(scale, x[k], g[k]);
  Group<__nv_bfloat16, VEC>::store(p, step, n, g);
}

// A part, past the first-level cache: another block may have written it.
template <bool VEC>
__device__ __forceinline__ void load_part(const float *p, int step, int n, float (&x)[8]) {
  if (VEC) {
    const float4 a = __ldcg(reinterpret_cast<const float4 *>(p)), b = __ldcg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? __ldcg(p + k * step) : 0.f;
  }
}

// A row that crosses tiles: its parts are those of tiles first .. last, the first one's second, the others' first.  Each
// warp counts its tile off once its part is written; the one that counts the last off adds them up in their order, up to
// kJoin of them.  Of a longer row the tiles of an aligned group of kJoin count among themselves, their sum takes the place
// of the group's first part, and the groups count in turn.
constexpr int kJoin = 16;  // 8192 x 2048 of one row 36.8 us, of 200 rows 28.8; 32: 35.6 and 28.9

// The tile in which the row that comes into `tile` begins: the last one before it that the row does not fill.  A lane
// looks at one tile's first place, 32 tiles at a time, or far from here at steps that narrow by 32.
__device__ __forceinline__ int begins_at(const SumArgs &a, int tile, int row) {
  const int lane = threadIdx.x & 31;
  // the row fills the tiles hi .. tile - 1 but for their last tokens' rows; it begins in lo .. hi
  int hi = tile, lo = 0;
  for (int step = 1;; step = max((hi - lo + 31) / 32, 1)) {
    const int t = hi - 1 - lane * step;  // whether the row is there before its first place
    const bool reaches = t >= 0 && t * a.tile > 0 && a.key[t * a.tile - 1] == row;
    const unsigned no = __ballot_sync(0xFFFFFFFFu, !reaches);
    const int first = __ffs(int(no)) - 1;  // -1: all 32 do
    if (first >= 0) {
      if (step == 1) return hi - 1 - first;
      lo = max(lo, hi - 1 - first * step);
      if (first > 0) hi = hi - 1 - (first - 1) * step;
    } else {
      hi = hi - 1 - 31 * step;
    }
  }
}

// The tile in which the row that goes on from `tile` ends.
__device__ __forceinline__ int ends_at(const SumArgs &a, int tile, int row) {
  const int lane = threadIdx.x & 31;
  int lo = tile, hi = a.tiles - 1;  // it ends in lo .. hi
  for (int step = 1;; step = max((hi - lo + 31) / 32, 1)) {
    const int t = lo + 1 + lane * step;  // whether the row goes on behind its last place
    const bool goes = t < a.tiles - 1 && a.key[(t + 1) * a.tile] == row;
    const unsigned no = __ballot_sync(0xFFFFFFFFu, !goes);
    const int first = __ffs(int(no)) - 1;
    if (first >= 0) {
      if (step == 1) return lo + 1 + first;
      hi = min(hi, lo + 1 + first * step);
      if (first > 0) lo = lo + 1 + (first - 1) * step;
    } else {
      lo = lo + 1 + 31 * step;
    }
  }
}

template <typename TG, bool VEC>
__device__ __forceinline__ void join_row(const SumArgs &a, int tile, int first, int last, int row, int group, int64_t c, int step,
                                         int n) {
  const int lane = threadIdx.x & 31;
  const auto place = [&](int t) { return a.part + (int64_t(t) * 2 + (t == first)) * a.cols + c; };
  const auto last_of = [&](int t, int which, int of) {  // whether this warp counts the last of them off
    __threadfence();
    __syncwarp();
    int before = 0;
    if (lane == 0) before = atomicAdd(a.counters + (int64_t(t) * 3 + which) * a.groups + group, 1);
    before = __shfl_sync(0xFFFFFFFFu, before, 0);
    __threadfence();
    return before == of - 1;
  };
  float acc[8];
  const auto sum = [&](int from, int to, int by, bool groups) {  // parts from .. to, four in flight
    constexpr int N = 4;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    for (int t0 = from; t0 <= to; t0 += N * by) {
      float x[N][8];
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = 0.f;
        const int t = t0 + i * by;
        if (t <= to && n > 0) load_part<VEC>(place(groups ? max(t, first) : t), step, n, x[i]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += x[i][k];
    }
  };
  TG *const grad = static_cast<TG *>(a.grad) + int64_t(row) * a.cols + c;
  if (last - first < kJoin) {
    if (!last_of(first, 1, last - first + 1)) return;
    sum(first, last, 1, false);
  } else {
    const int g = tile & ~(kJoin - 1), t0 = max(first, g), t1 = min(last, g + kJoin - 1);
    if (!last_of(t0, t0 == first, t1 - t0 + 1)) return;
    sum(t0, t1, 1, false);
    if (n > 0) Group<float, VEC>::store(place(t0), step, n, acc);
    if (!last_of(first, 2, last / kJoin - first / kJoin + 1)) return;
    sum(first & ~(kJoin - 1), last, kJoin, true);
  }
  if (n > 0) add8<VEC>(grad, step, n, a.scale, acc);
}

// A tile a thread row (whole warps, so that a warp's lanes read the keys of 32 places at once and hand them round), eight
// columns a thread, kFlight tokens' rows in flight.  Bound by the chain keys, rows, parts, counters, joined rows, and by
// the gradient's lines, which the L2 has to fetch: [8192, 2048] bf16 of 32000 rows into fp32 50 us together with the sort
// (22 us of bytes; eight in flight at two blocks an SM 53).
constexpr int kFlight = 4;

template <typename TD, typename TG, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_sum_kernel(const __grid_constant__ SumArgs a) {
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  int64_t c;
  int n = 0;
  const int tile = int(blockIdx.y) * blockDim.y + threadIdx.y, lane = threadIdx.x & 31;
  const bool mine = columns<VEC>(a.cols, c, n);
  if (!mine) n = 0;
  if (tile >= a.tiles) return;  // the whole warp
  const int tx = blockDim.x, rows = int(a.rows);
  const int p0 = tile * a.tile, p1 = min(p0 + a.tile, a.tokens);
  const int after = p1 < a.tokens ? a.key[p1] : rows, before = p0 > 0 ? a.key[p0 - 1] : -1;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  float *const part = a.part + int64_t(tile) * 2 * a.cols + c;
  const int group = int(blockIdx.x) * (tx >> 5) + (int(threadIdx.x) >> 5);
  int row = rows, came = rows;  // the row being summed; the one that came in, once its part is written
  bool open = false;            // the row being summed came in from the tile before
  for (int q0 = p0; q0 < p1; q0 += 32) {
    const int q = q0 + lane;
    const int key = q < p1 ? a.key[q] : rows, token = q < p1 ? a.token[q] : 0;  // not a token where key is rows
    if (q0 == p0) {
      row = __shfl_sync(0xFFFFFFFFu, key, 0);
      if (row >= rows) return;  // behind the shard's tokens
      open = before == row;
    }
    for (int i0 = 0; i0 < min(32, p1 - q0); i0 += kFlight) {
      Group<TD, VEC> x[kFlight];
      int k[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        k[i] = __shfl_sync(0xFFFFFFFFu, key, i0 + i);
        const int t = __shfl_sync(0xFFFFFFFFu, token, i0 + i);
        if (k[i] < rows && mine) x[i].load(static_cast<const TD *>(a.dout) + int64_t(t) * a.dout_ld + c, tx, n);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (k[i] >= rows) continue;
        if (k[i] != row) {
          if (open) {
            if (mine) Group<float, VEC>::store(part, tx, n, acc);
            came = row;
          } else if (mine) {
            add8<VEC>(static_cast<TG *>(a.grad) + int64_t(row) * a.cols + c, tx, n, a.scale, acc);
          }
          open = false;
          row = k[i];
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        }
        if (!mine) continue;
        float f[8];
        x[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += f[j];
      }
    }
  }
  const bool goes = after == row;
  if (mine) {
    if (open) Group<float, VEC>::store(part, tx, n, acc);
    else if (goes) Group<float, VEC>::store(part + a.cols, tx, n, acc);
    else add8<VEC>(static_cast<TG *>(a.grad) + int64_t(row) * a.cols + c, tx, n, a.scale, acc);
  }
  const bool came_in = came < rows;
  if (!came_in && !open && !goes) return;
  const int begins = came_in || open ? begins_at(a, tile, came_in ? came : row) : tile, ends = goes ? ends_at(a, tile, row) : tile;
  if (came_in) join_row<TG, VEC>(a, tile, begins, tile, came, group, c, tx, n);
  if (open || goes) join_row<TG, VEC>(a, tile, open ? begins : tile, ends, row, group, c, tx, n);
}

// So few tokens that every block sorts them for itself, by counting: no second launch and no parts, a row's tokens are
// summed where its first place's tile is.  64 tokens x 2048 take 5.2 us (two launches 7.6), 10.0 where all are one row's
// (9.6); at 128 one row's take 19.4 and 10.7.
constexpr int kFewTokens = 64, kFewTile = 4;

struct FewArgs {
  const void *ids, *dout;
  void *grad;
  int64_t dout_ld, first_row, rows, cols;
  int32_t tokens, wide;
  float scale;
};

template <typename TD, typename TG, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int F = VEC ? 8 : 4;  // tokens' rows in flight
  __shared__ int32_t seen[kFewTokens], key[kFewTokens + 1], token[kFewTokens];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int me = threadIdx.y * blockDim.x + threadIdx.x, T = a.tokens, rows = int(a.rows);
  for (int t = me; t < T; t += kThreads) seen[t] = int32_t(row_of(a.ids, a.wide, t, a.first_row, a.rows));
  if (me == 0) key[T] = rows;
  __syncthreads();
  for (int t = me; t < T; t += kThreads) {
    const int32_t k = seen[t];
    int place = 0;
    for (int s = 0; s < T; ++s) place += seen[s] < k || (seen[s] == k && s < t);
    key[place] = k;
    token[place] = t;
  }
  __syncthreads();
  int64_t c;
  int n;
  if (!columns<VEC>(a.cols, c, n)) return;
  const int p0 = (int(blockIdx.y) * blockDim.y + threadIdx.y) * kFewTile, p1 = min(p0 + kFewTile, T), tx = blockDim.x;
  for (int p = p0; p < p1;) {
    const int32_t row = key[p];
    if (row >= rows) return;
    int end = p + 1;
    while (key[end] == row) ++end;
    if (p > 0 && key[p - 1] == row) {  // begun before this tile
      p = end;
      continue;
    }
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    for (int q = p; q < end; q += F) {
      Group<TD, VEC> x[F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        x[i].clear();
        if (q + i < end) x[i].load(static_cast<const TD *>(a.dout) + int64_t(token[q + i]) * a.dout_ld + c, tx, n);
      }
#pragma unroll
      for (int i = 0; i < F; ++i) {
        float f[8];
        x[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += f[j];
      }
    }
    add8<VEC>(static_cast<TG *>(a.grad) + int64_t(row) * a.cols + c, tx, n, a.scale, acc);
    p = end;
  }
}

// --------------------------------------------------------------------------- host

constexpr int64_t kMaxDim = int64_t(1) << 30;

// Threads a block across a row's groups of eight (at least `least`), and rows of such threads.
dim3 block_of(int64_t cols, int least) {
  int tx = least;
  while (tx < kThreads && 8 * tx < cols) tx *= 2;
  return dim3(tx, kThreads / tx);
}

// Whether every row starts on eight elements' own size.
bool in_eights(const void *p, int64_t ld, int64_t es) {
  return (reinterpret_cast<uintptr_t>(p) & uintptr_t(8 * es - 1)) == 0 && ld % 8 == 0;
}

int64_t size_of(int dt) { return dt == GTP_F32 ? 4 : 2; }
bool float_type(int dt) { return dt == GTP_F32 || dt == GTP_BF16; }

gtp_status check_sizes(int64_t tokens, int64_t first_row, int64_t rows, int64_t cols, int32_t ids64) {
  if (tokens < 0 || rows < 0 || cols < 0 || first_row < 0) return gtp::fail(GTP_E_ARG, "negative size");
  if (ids64 != 0 && ids64 != 1) return gtp::fail(GTP_E_ARG, "ids64 must be 0 or 1");
  if (tokens > kMaxDim || rows > kMaxDim || cols > kMaxDim) return gtp::fail(GTP_E_SHAPE, "a dimension above 2^30");
  const int64_t c = std::max<int64_t>(cols, 1);
  if (tokens > (int64_t(1) << 40) / c || rows > (int64_t(1) << 40) / c)
    return gtp::fail(GTP_E_SHAPE, "more than 2^40 elements");
  return GTP_OK;
}

gtp_status check_ld(const char *name, int64_t ld, int64_t n, int64_t cols) {
  if (n > 1 && ld < cols) return gtp::fail(GTP_E_ARG, "a row stride of %s below cols", name);
  if (n > 1 && ld > (int64_t(1) << 50) / n) return gtp::fail(GTP_E_SHAPE, "%s spans more than 2^50 elements", name);
  return GTP_OK;
}

gtp::ByteRange span_of(const void *p, int64_t n, int64_t ld, int64_t cols, int64_t es) {
  return gtp::byte_range(p, n && cols ? ((n - 1) * ld + cols) * es : 0);
}

template <typename TI, typename TO>
gtp_status launch_lookup(const LookupArgs &a, const gtp::DeviceInfo &dev, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && in_eights(a.table, a.table_ld, sizeof(TI)) && in_eights(a.out, a.out_ld, sizeof(TO));
  const dim3 block = block_of(a.cols, 1);
  const int64_t gx = (a.cols + 8 * block.x - 1) / (8 * block.x), fill = std::max<int64_t>(1, int64_t(dev.sm_count) * 8 / gx);
  const int64_t rows = (a.tokens + block.y - 1) / block.y;  // of blocks, at a token a thread
  // tokens a thread: four of whole vectors ([8192, 2048] bf16 12.8 us, 5.2 TB/s; one at a time 15.2), one of single elements
  // ([8192, 2047] 25.2 us, two 25.5, four 26.9; into fp32 26.4 and 27.5); few tokens one at a time, spread over the machine
  const bool many = vec && rows > fill;
  const int n = many ? 4 : 1;
  const dim3 grid(unsigned(gx), unsigned(std::min<int64_t>((rows + n - 1) / n, 65535)));
  const auto kernel = many  ? embedding_kernel<TI, TO, true, 4>
                      : vec ? embedding_kernel<TI, TO, true, 1>
                            : embedding_kernel<TI, TO, false, 1>;
  return gtp::launch_overlapped(kernel, grid, block, 0, st, "embedding", a);
}

struct GradPlan {
  int32_t tile, tiles, sort_tiles;
  bool radix;
  int32_t groups;
  int64_t key, token, key2, token2, counts, counters, part, bytes;  // places in the workspace
};

// Tokens a thread of a sort tile: few where that keeps the tiles in kFewTiles (16384 x 256: 30 us with 2, 37 with 8), else
// more, so that their counts stay few (65536: 75 us with 2, 47 with 8).
int rounds_of(int64_t tokens) { return tokens <= 2 * kTileThreads * kFewTiles ? 2 : 8; }

GradPlan grad_plan(int64_t tokens, int64_t rows, int64_t cols) {
  GradPlan p = {};
  p.radix = tokens > kRankMost || rows * tokens >= (int64_t(1) << 32) - 1;
  // tiles: short ones spread few tokens over the machine, and longer ones keep the parts few from 4096 tiles on.  Eight
  // tokens: [8192, 2048] that are all one row's 37 us, of 200 rows 29; with tiles of four 52 and 37 (but [2048, 256] 15.1 and
  // 12.6)
  p.tile = int32_t(std::max<int64_t>(8, (tokens + 4095) / 4096));
  p.tiles = int32_t((tokens + p.tile - 1) / p.tile);
  const int64_t each = kTileThreads * rounds_of(tokens);
  p.sort_tiles = int32_t((tokens + each - 1) / each);
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) & ~int64_t(255);
    return here;
  };
  p.key = take(4 * tokens);
  p.token = take(4 * tokens);
  if (p.radix) {
    p.key2 = take(4 * tokens);
    p.token2 = take(4 * tokens);
    p.counts = take(int64_t(4) * 256 * p.sort_tiles);
  }
  const dim3 block = block_of(cols, 32);
  p.groups = int32_t((cols + 8 * block.x - 1) / (8 * block.x) * (block.x / 32));
  p.counters = take(int64_t(12) * p.tiles * p.groups);
  p.part = take(int64_t(8) * p.tiles * cols);
  p.bytes = at;
  return p;
}

gtp_status sort_tokens(SortArgs &a, const GradPlan &plan, cudaStream_t st) {
  if (!plan.radix) {
    const size_t smem = size_t((a.tokens + 3) & ~3) * 4;
    return gtp::launch_overlapped(rank_kernel, unsigned((a.tokens + kOwn - 1) / kOwn), kRankThreads, smem, st, "embedding_grad",
                                  a);
  }
  int bits = 1;  // of the keys 0 .. rows
  while (bits < 31 && (int64_t(1) << bits) <= a.rows) ++bits;
  const int passes = (bits + 7) / 8;
  a.scan = a.tiles > kFewTiles;
  const bool wide = rounds_of(a.tokens) == 8;
  const int32_t *key = nullptr, *token = nullptr;
  for (int i = 0; i < passes; ++i) {  // the last pass writes the result
    const bool into_first = (passes - 1 - i) % 2 == 0;
    int32_t *key_out = into_first ? a.key : a.key2, *token_out = into_first ? a.token : a.token2;
    gtp_status s = gtp::launch_overlapped(wide ? radix_count_kernel<8> : radix_count_kernel<2>, unsigned(a.tiles), kTileThreads, 0, st,
                                          "embedding_grad", a, key, 8 * i);
    if (!s && a.scan) s = gtp::launch_overlapped(radix_scan_kernel, 1, kScanThreads, 0, st, "embedding_grad", a);
    if (!s)
      s = gtp::launch_overlapped(a.scan ? radix_scatter_kernel<8, true>
                                 : wide ? radix_scatter_kernel<8, false>
                                        : radix_scatter_kernel<2, false>,
                                 unsigned(a.tiles), kTileThreads, 0, st, "embedding_grad", a, key, token, key_out, token_out, 8 * i);
    if (s) return s;
    key = key_out, token = token_out;
  }
  return GTP_OK;
}

template <typename TD, typename TG>
gtp_status launch_sums(const SumArgs &a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && in_eights(a.dout, a.dout_ld, sizeof(TD)) && in_eights(a.grad, a.cols, sizeof(TG));
  const dim3 block = block_of(a.cols, 32);
  const dim3 grid(unsigned((a.cols + 8 * block.x - 1) / (8 * block.x)), (a.tiles + block.y - 1) / block.y);
  return gtp::launch_overlapped(vec ? embedding_sum_kernel<TD, TG, true> : embedding_sum_kernel<TD, TG, false>, grid, block, 0, st,
                                "embedding_grad", a);
}

template <typename TD, typename TG>
gtp_status launch_few(const FewArgs &a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && in_eights(a.dout, a.dout_ld, sizeof(TD)) && in_eights(a.grad, a.cols, sizeof(TG));
  const dim3 block = block_of(a.cols, 32);
  const int tiles = (a.tokens + kFewTile - 1) / kFewTile;
  const dim3 grid(unsigned((a.cols + 8 * block.x - 1) / (8 * block.x)), (tiles + block.y - 1) / block.y);
  return gtp::launch_overlapped(vec ? embedding_few_kernel<TD, TG, true> : embedding_few_kernel<TD, TG, false>, grid, block, 0, st,
                                "embedding_grad", a);
}

}  // namespace

extern "C" gtp_status gtp_embedding(const gtp_embedding_desc *d, gtp_stream stream) {
  gtp::clear_error();
  if (!d) return gtp::fail(GTP_E_ARG, "null descriptor");
  if (d->reserved) return gtp::fail(GTP_E_ARG, "reserved must be 0");
  if (!float_type(d->table_dtype) || !float_type(d->out_dtype)) return gtp::fail(GTP_E_DTYPE, "dtypes must be F32 or BF16");
  const int64_t T = d->tokens, R = d->rows, C = d->cols;
  if (gtp_status s = check_sizes(T, d->first_row, R, C, d->ids64)) return s;
  if (gtp_status s = check_ld("table", d->table_ld, R, C)) return s;
  if (gtp_status s = check_ld("out", d->out_ld, T, C)) return s;
  if (T == 0 || C == 0) return GTP_OK;
  if (!d->ids || !d->out || (!d->table && R)) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t ts = size_of(d->table_dtype), os = size_of(d->out_dtype), is = d->ids64 ? 8 : 4;
  if ((reinterpret_cast<uintptr_t>(d->ids) & uintptr_t(is - 1)) || (reinterpret_cast<uintptr_t>(d->table) & uintptr_t(ts - 1)) ||
      (reinterpret_cast<uintptr_t>(d->out) & uintptr_t(os - 1)))
    return gtp::fail(GTP_E_ALIGN, "arrays must be aligned to their elements");
  const int64_t table_ld = R > 1 ? d->table_ld : C, out_ld = T > 1 ? d->out_ld : C;
  const gtp::ByteRange o = span_of(d->out, T, out_ld, C, os);
  if (gtp::overlap(o, span_of(d->table, R, table_ld, C, ts)) || gtp::overlap(o, gtp::byte_range(d->ids, T * is)))
    return gtp::fail(GTP_E_ARG, "out overlaps an input");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  const LookupArgs a = {d->ids, d->table, d->out, T, table_ld, out_ld, d->first_row, R, C, d->scale, d->ids64};
  cudaStream_t st = gtp::as_stream(stream);
  using B = __nv_bfloat16;
  if (d->table_dtype == GTP_F32)
    return d->out_dtype == GTP_F32 ? launch_lookup<float, float>(a, dev, st) : launch_lookup<float, B>(a, dev, st);
  return d->out_dtype == GTP_F32 ? launch_lookup<B, float>(a, dev, st) : launch_lookup<B, B>(a, dev, st);
}

extern "C" int64_t gtp_embedding_grad_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols) {
  if (check_sizes(tokens, 0, rows, cols, 0)) return -1;
  if (tokens == 0 || rows == 0 || cols == 0) return 0;
  return grad_plan(tokens, rows, cols).bytes;
}

extern "C" gtp_status gtp_embedding_grad_accum(const gtp_embedding_grad_desc *d, void *workspace, int64_t workspace_bytes,
                                               gtp_stream stream) {
  gtp::clear_error();
  if (!d) return gtp::fail(GTP_E_ARG, "null descriptor");
  if (d->reserved) return gtp::fail(GTP_E_ARG, "reserved must be 0");
  if (!float_type(d->dout_dtype) || !float_type(d->grad_dtype)) return gtp::fail(GTP_E_DTYPE, "dtypes must be F32 or BF16");
  const int64_t T = d->tokens, R = d->rows, C = d->cols;
  if (gtp_status s = check_sizes(T, d->first_row, R, C, d->ids64)) return s;
  if (gtp_status s = check_ld("dout", d->dout_ld, T, C)) return s;
  if (d->grad_offset < 0 || d->grad_numel_total < 0 || d->grad_numel_total > (int64_t(1) << 50) ||
      d->grad_offset > d->grad_numel_total || R * C > d->grad_numel_total - d->grad_offset)
    return gtp::fail(GTP_E_RANGE, "the view of %lld elements at %lld leaves a buffer of %lld", (long long)(R * C),
                     (long long)d->grad_offset, (long long)d->grad_numel_total);
  if (T == 0 || R == 0 || C == 0) return GTP_OK;
  if (!d->ids || !d->dout || !d->grad_data || !workspace) return gtp::fail(GTP_E_ARG, "null pointer");
  const int64_t ds = size_of(d->dout_dtype), gs = size_of(d->grad_dtype), is = d->ids64 ? 8 : 4;
  if ((reinterpret_cast<uintptr_t>(d->ids) & uintptr_t(is - 1)) || (reinterpret_cast<uintptr_t>(d->dout) & uintptr_t(ds - 1)) ||
      (reinterpret_cast<uintptr_t>(d->grad_data) & uintptr_t(gs - 1)))
    return gtp::fail(GTP_E_ALIGN, "arrays must be aligned to their elements");
  if (reinterpret_cast<uintptr_t>(workspace) & 31u) return gtp::fail(GTP_E_ALIGN, "workspace must be 32-byte aligned");
  const GradPlan plan = grad_plan(T, R, C);
  if (workspace_bytes < plan.bytes)
    return gtp::fail(GTP_E_CAPACITY, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)plan.bytes);
  const int64_t dout_ld = T > 1 ? d->dout_ld : C;
  char *const grad = static_cast<char *>(d->grad_data) + d->grad_offset * gs, *const ws = static_cast<char *>(workspace);
  const gtp::ByteRange g = gtp::byte_range(grad, R * C * gs), w = gtp::byte_range(ws, plan.bytes),
                       x = span_of(d->dout, T, dout_ld, C, ds), i = gtp::byte_range(d->ids, T * is);
  if (gtp::overlap(g, x) || gtp::overlap(g, i) || gtp::overlap(w, x) || gtp::overlap(w, i) || gtp::overlap(w, g))
    return gtp::fail(GTP_E_ARG, "the gradient view or the workspace overlaps an input or the other");
  gtp::DeviceInfo dev;
  if (gtp_status s = gtp::require_sm103(&dev)) return s;
  cudaStream_t st = gtp::as_stream(stream);
  using B = __nv_bfloat16;
  if (T <= kFewTokens) {
    const FewArgs a = {d->ids, d->dout, grad, dout_ld, d->first_row, R, C, int32_t(T), d->ids64, d->scale};
    if (d->dout_dtype == GTP_F32) return d->grad_dtype == GTP_F32 ? launch_few<float, float>(a, st) : launch_few<float, B>(a, st);
    return d->grad_dtype == GTP_F32 ? launch_few<B, float>(a, st) : launch_few<B, B>(a, st);
  }
  const auto at = [&](int64_t place) { return reinterpret_cast<int32_t *>(ws + place); };
  SortArgs sort = {};
  sort.ids = d->ids, sort.first_row = d->first_row, sort.rows = R, sort.tokens = int32_t(T), sort.wide = d->ids64;
  sort.key = at(plan.key), sort.token = at(plan.token), sort.key2 = at(plan.key2), sort.token2 = at(plan.token2);
  sort.counts = at(plan.counts), sort.tiles = plan.sort_tiles;
  sort.counters = at(plan.counters), sort.counter_count = int64_t(3) * plan.tiles * plan.groups;
  if (gtp_status s = sort_tokens(sort, plan, st)) return s;
  SumArgs a = {};
  a.key = sort.key, a.token = sort.token, a.dout = d->dout, a.grad = grad, a.part = reinterpret_cast<float *>(ws + plan.part);
  a.counters = sort.counters, a.groups = plan.groups;
  a.dout_ld = dout_ld, a.rows = R, a.cols = C, a.tokens = int32_t(T), a.tile = plan.tile, a.tiles = plan.tiles, a.scale = d->scale;
  if (d->dout_dtype == GTP_F32) return d->grad_dtype == GTP_F32 ? launch_sums<float, float>(a, st) : launch_sums<float, B>(a, st);
  return d->grad_dtype == GTP_F32 ? launch_sums<B, float>(a, st) : launch_sums<B, B>(a, st);
}
