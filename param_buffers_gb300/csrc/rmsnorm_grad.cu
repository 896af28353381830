// The gradient of the root-mean-square norm (rmsnorm.cu), the weight's accumulated into the flat gradient buffer.
//
// Pages: "Megatron-LM architecture and source guide" (arganzheng.life), §1 (the norms of a transformer layer);
// "05 · grad/param buffer ..." (llm-infra-atlas), §5 (main_grad as a view of the flat buffer).
//
//   n = s r, g = dy w:   dx = r (g - n mean(g n)) + dsum                    dw += sum over rows of dy n
// Sums in fp32, in an order that the sizes alone decide: every place's rows leave a part of dw, a second kernel adds the
// parts up.  Bound by the bytes of dy, s, dsum and dx.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "device.h"
#include "eight.cuh"
#include "norm_args.h"
#include "sm100_ptx.cuh"

namespace gtp {
void clear_error();
}

namespace {

constexpr int kRowThreads = 512;  // of a row, at most
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxCols = 32 * kRowThreads;

// --------------------------------------------------------------------------- gradient

struct GradArgs {
  const void *dy, *sum, *weight, *dsum;
  const float *rstd;
  void *dx;
  float *part;  // [gridDim.x * blockDim.y][cols]: the weight's gradient of each place's rows
  int64_t rows, cols, dy_ld, sum_ld, dsum_ld, dx_ld;
  float inv_cols;
  int weight_f32;
};

using gtp::Eight;
using gtp::warp_sum;

// Sums of N rows at a time over a row's threads, as the forward's.
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

// A thread keeps its columns (V groups of eight) over all its rows, so that their part of the weight's gradient, and with
// one group the weight, stay in registers.  N rows at a time have all their loads in flight together, as they lie in
// memory, and share a barrier; what is between the loads and the outputs is computed twice rather than kept.
template <typename TD, typename TS, int V, int N>
__global__ void __launch_bounds__(kRowThreads) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float part[2][N][32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int tx = blockDim.x;
  float w[8], dw[V][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    w[k] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) dw[v][k] = 0.f;
  }
  const auto column = [&](int v) { return 8 * (int64_t(v) * tx + threadIdx.x); };
  if (V == 1 && column(0) < a.cols) gtp::load8_of(a.weight, a.weight_f32, column(0), w);
  int flip = 0;
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < a.rows; r0 += N * step, flip ^= 1) {
    Eight<TD> dy[N][V];
    Eight<TS> s[N][V], ds[N][V];
    float r[N], dot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = r0 + i * step + threadIdx.y;
      r[i] = row < a.rows ? a.rstd[row] : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        dy[i][v].clear();
        s[i][v].clear();
        ds[i][v].clear();
        if (row < a.rows && column(v) < a.cols) {
          dy[i][v].load(static_cast<const TD *>(a.dy) + row * a.dy_ld + column(v));
          s[i][v].load(static_cast<const TS *>(a.sum) + row * a.sum_ld + column(v));
          if (a.dsum) ds[i][v].load(static_cast<const TS *>(a.dsum) + row * a.dsum_ld + column(v));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dot[i] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (V > 1 && column(v) < a.cols) gtp::load8_of(a.weight, a.weight_f32, column(v), w);
        float g[8], n[8];
        dy[i][v].get(g);
        s[i][v].get(n);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          n[k] *= r[i];
          dw[v][k] = fmaf(g[k], n[k], dw[v][k]);
          dot[i] = fmaf(g[k] * w[k], n[k], dot[i]);
        }
      }
    }
    row_sums<N>(dot, part, flip);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (V > 1 && column(v) < a.cols) gtp::load8_of(a.weight, a.weight_f32, column(v), w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t row = r0 + i * step + threadIdx.y;
        if (row >= a.rows || column(v) >= a.cols) continue;
        const float mean = dot[i] * a.inv_cols;
        float g[8], n[8], d[8];
        dy[i][v].get(g);
        s[i][v].get(n);
        ds[i][v].get(d);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = fmaf(r[i], fmaf(-(n[k] * r[i]), mean, g[k] * w[k]), d[k]);
        Eight<TS> out;
        out.set(d);
        out.store(static_cast<TS *>(a.dx) + row * a.dx_ld + column(v));
      }
    }
  }
  float *const out = a.part + (int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * a.cols;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (column(v) < a.cols) {
      Eight<float> e;
      e.set(dw[v]);
      e.store(out + column(v));
    }
}

// Rows that start anywhere: the elements TX apart are a thread's (as the forward's).
template <typename TD, typename TS, int TX, int K>
__global__ void __launch_bounds__(TX == 32 ? 256 : TX, TX == 32 ? 3 : 1024 / TX) norm_grad_elements_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float part[2][1][32];
  gtp::ptx::allow_dependents();
  gtp::ptx::wait_prior_grid();
  const int cols = int(a.cols), t = threadIdx.x;
  // the weight in registers, and elements as they lie in memory, so that all loads are under way together ([8192, 2047] bf16 38.5
  // us, converted one by one 55); of sixteen fp32 elements the registers do not hold that ([4096, 16001] all fp32 336 us, so 384;
  // bf16 239, one by one 287)
  constexpr bool KEEP = K <= 8 || sizeof(TD) + 2 * sizeof(TS) < 12;
  float w[KEEP ? K : 1], dw[K];
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k] = 0.f;
  if constexpr (KEEP) gtp::load_apart_of<TX>(a.weight, a.weight_f32, t, cols, w);
  int flip = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < a.rows; r0 += int64_t(gridDim.x) * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < a.rows;
    const float r = live ? a.rstd[row] : 0.f;
    const TD *const dy = static_cast<const TD *>(a.dy) + row * a.dy_ld + t;
    const TS *const s = static_cast<const TS *>(a.sum) + row * a.sum_ld + t;
    const TS *const ds = static_cast<const TS *>(a.dsum) + (a.dsum ? row * a.dsum_ld + t : 0);
    float g[K], n[K], dot[1] = {0.f};
    TS d[K];  // loaded with the others, not behind the stores
    if constexpr (KEEP) {
      TD dy_in[K];
      TS s_in[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool there = live && t + k * TX < cols;
        dy_in[k] = there ? dy[k * TX] : TD(0.f);
        s_in[k] = there ? s[k * TX] : TS(0.f);
        d[k] = there && a.dsum ? ds[k * TX] : TS(0.f);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) g[k] = float(dy_in[k]), n[k] = float(s_in[k]);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) g[k] = live && t + k * TX < cols ? gtp::load1(dy + k * TX) : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) n[k] = live && t + k * TX < cols ? gtp::load1(s + k * TX) : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) d[k] = live && a.dsum && t + k * TX < cols ? ds[k * TX] : TS(0.f);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float wk = KEEP ? w[KEEP ? k : 0] : t + k * TX < cols ? gtp::load1_of(a.weight, a.weight_f32, t + k * TX) : 0.f;
      n[k] *= r;
      dw[k] = fmaf(g[k], n[k], dw[k]);
      g[k] *= wk;
      dot[0] = fmaf(g[k], n[k], dot[0]);
    }
    row_sums<1>(dot, part, flip);
    if (!live) continue;
    const float mean = dot[0] * a.inv_cols;
    TS *const dx = static_cast<TS *>(a.dx) + row * a.dx_ld + t;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t + k * TX < cols) gtp::store1(dx + k * TX, fmaf(r, fmaf(-n[k], mean, g[k]), gtp::load1(&d[k])));
  }
  float *const out = a.part + (int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * a.cols + t;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (t + k * TX < cols) out[k * TX] = dw[k];
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
    constexpr int N = 8;  // parts in flight
    for (int p0 = threadIdx.y; p0 < parts; p0 += 32 * N) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = p0 + 32 * i < parts ? part[int64_t(p0 + 32 * i) * cols + c] : 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) s += v[i];
    }
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(sums[threadIdx.x][threadIdx.y]);  // warp y: column y of the block
  const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < cols) gtp::store1(grad + col, gtp::load1(grad + col) + s);
}

// --------------------------------------------------------------------------- host

// Threads a row, rows a block, groups of eight a thread (one up to 4096 columns, else four: [8192, 4096] bf16 53.9 and 57.4
// us, [8192, 2048] 29.2 and 36.2) and blocks: those that run at once, 512 threads an SM (128 registers each).  One rule for
// the workspace's size and the launch.
struct GradShape {
  int tx, ty, V, grid;
};

GradShape grad_shape(int64_t rows, int64_t cols, int sms) {
  const int64_t groups = (cols + 7) / 8;
  const int V = groups <= kRowThreads ? 1 : 4;
  const int tx = int((groups + 32 * V - 1) / (32 * V)) * 32, ty = tx == 32 ? 8 : 1;
  const int64_t most = int64_t(sms) * std::max(1, 512 / (tx * ty));
  return {tx, ty, V, int(std::min<int64_t>((rows + ty - 1) / ty, most))};
}

// The same for rows that start anywhere: 1024 threads an SM of 64 registers each, 768 where a warp has a row ([8192, 250]
// 26.4 us).
GradShape elements_shape(int64_t rows, int64_t cols, int sms) {
  const int tx = cols <= 32 * 8 ? 32 : cols <= 256 * 8 ? 256 : cols <= 512 * 8 ? 512 : 1024, ty = tx == 32 ? 8 : 1;
  const int64_t most = int64_t(sms) * (tx == 32 ? 3 : 1024 / tx);
  return {tx, ty, cols <= 1024 * 8 ? 1 : 2, int(std::min<int64_t>((rows + ty - 1) / ty, most))};
}

constexpr int kMostSms = 160;  // the workspace's size is asked for without a device: at least an sm_103 GPU's SMs

template <typename TD, typename TS>
gtp_status launch_grad(const GradArgs &a, bool vec, const GradShape &s, cudaStream_t st) {
  constexpr int N = sizeof(TD) + 2 * sizeof(TS) > 6 ? 2 : 4;
  void (*kernel)(GradArgs);
  if (vec) kernel = s.V == 1 ? norm_grad_kernel<TD, TS, 1, N> : norm_grad_kernel<TD, TS, 4, 1>;
  else
    kernel = s.tx == 32 ? norm_grad_elements_kernel<TD, TS, 32, 8>
             : s.tx == 256 ? norm_grad_elements_kernel<TD, TS, 256, 8>
             : s.tx == 512 ? norm_grad_elements_kernel<TD, TS, 512, 8>
             : s.V == 1    ? norm_grad_elements_kernel<TD, TS, 1024, 8> : norm_grad_elements_kernel<TD, TS, 1024, 16>;
  return gtp::launch_overlapped(kernel, unsigned(s.grid), dim3(s.tx, s.ty), 0, st, "rmsnorm_grad", a);
}

}  // namespace

extern "C" int64_t gtp_rmsnorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxCols) return -1;
  if (rows == 0 || cols == 0) return 0;
  const GradShape v = grad_shape(rows, cols, kMostSms), e = elements_shape(rows, cols, kMostSms);
  return int64_t(std::max(v.grid * v.ty, e.grid * e.ty)) * cols * 4;
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
  if (!aligned(d->rstd, 4) || !aligned(d->grad_data, gs) || !aligned(workspace, 32))
    return gtp::fail(GTP_E_ALIGN, "rstd and grad_data must be aligned to their elements, the workspace to 32 bytes");
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
  a.inv_cols = 1.f / float(C);
  const int sms = std::min(dev.sm_count, kMostSms);
  const GradShape shape = vec ? grad_shape(R, C, sms) : elements_shape(R, C, sms);
  cudaStream_t st = gtp::as_stream(stream);
  using B = __nv_bfloat16;
  gtp_status e;
  if (d->dy_dtype == GTP_F32)
    e = d->sum_dtype == GTP_F32 ? launch_grad<float, float>(a, vec, shape, st) : launch_grad<float, B>(a, vec, shape, st);
  else
    e = d->sum_dtype == GTP_F32 ? launch_grad<B, float>(a, vec, shape, st) : launch_grad<B, B>(a, vec, shape, st);
  if (e) return e;
  const unsigned grid = unsigned((C + 31) / 32);
  const int parts = shape.grid * shape.ty;
  if (d->grad_dtype == GTP_F32)
    return gtp::launch_overlapped(norm_weight_kernel<float>, grid, dim3(32, 32), 0, st, "rmsnorm_grad",
                                  static_cast<const float *>(a.part), parts, C, reinterpret_cast<float *>(grad));
  return gtp::launch_overlapped(norm_weight_kernel<B>, grid, dim3(32, 32), 0, st, "rmsnorm_grad",
                                static_cast<const float *>(a.part), parts, C, reinterpret_cast<B *>(grad));
}

