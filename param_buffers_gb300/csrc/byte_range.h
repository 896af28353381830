// The bytes an argument spans, for the checks that outputs share none with inputs or each other.
#pragma once
#include <algorithm>
#include <cstdint>

namespace gtp {

struct ByteRange {
  uintptr_t begin, end;
};

inline ByteRange byte_range(const void *p, int64_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + uintptr_t(bytes)};
}

inline bool overlap(const ByteRange &a, const ByteRange &b) {
  return a.begin < a.end && b.begin < b.end && a.begin < b.end && b.begin < a.end;
}

// Runs of `bytes` bytes on a grid of up to three strides (bytes), the rows of a strided matrix or the heads of a tensor.
struct Runs {
  uintptr_t begin;
  int64_t bytes;
  struct Dim {
    int64_t stride, n;
  } dim[3];
};

// Whether the places a + sum k_i stride_i, |k_i| < n_i, come within (-below, above) of 0.  dim: strides descending, each no
// less than the smaller ones and a run span together, so that at every level two k_i are in question.
inline bool comes_near(int64_t a, int64_t below, int64_t above, const Runs::Dim *dim, int dims) {
  if (dims == 0) return -below < a && a < above;
  if (dim->n == 1) return comes_near(a, below, above, dim + 1, dims - 1);
  const int64_t s = dim->stride, q = -a / s, low = q - (-a % s < 0 ? 1 : 0);  // floor(-a / s)
  for (int64_t k = low; k <= low + 1; ++k)
    if (k > -dim->n && k < dim->n && comes_near(a + k * s, below, above, dim + 1, dims - 1)) return true;
  return false;
}

// Whether a run of `out` shares a byte with one of `in`; out's own runs are apart, nested as comes_near wants them.  Runs on
// the same strides (columns of one buffer, heads of one packed tensor) are compared exactly, others by what they span.
inline bool overlap(const Runs &out, const Runs &in) {
  int64_t span_out = out.bytes, span_in = in.bytes;
  bool alike = true;
  for (int i = 0; i < 3; ++i) {
    span_out += (out.dim[i].n - 1) * out.dim[i].stride;
    span_in += (in.dim[i].n - 1) * in.dim[i].stride;
    alike = alike && out.dim[i].n == in.dim[i].n && (out.dim[i].n == 1 || out.dim[i].stride == in.dim[i].stride);
  }
  if (out.begin >= in.begin + uintptr_t(span_in) || in.begin >= out.begin + uintptr_t(span_out)) return false;
  if (!alike) return true;
  Runs::Dim dim[3] = {out.dim[0], out.dim[1], out.dim[2]};
  std::sort(dim, dim + 3, [](const Runs::Dim &a, const Runs::Dim &b) { return a.stride > b.stride; });
  return comes_near(int64_t(in.begin - out.begin), in.bytes, out.bytes, dim, 3);
}

}  // namespace gtp
