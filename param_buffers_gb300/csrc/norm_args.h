// The norm's and its gradient's checks of their arguments.
#pragma once
#include <cstdint>

#include "byte_range.h"
#include "device.h"

namespace {

int64_t size_of(int dt) { return dt == GTP_F32 ? 4 : 2; }
bool float_type(int dt) { return dt == GTP_F32 || dt == GTP_BF16; }
bool aligned(const void *p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(to - 1)) == 0; }

struct Matrix {
  const char *name;
  const void *p;
  int64_t ld;
  int dt;
};

gtp_status check_matrix(const Matrix &m, int64_t rows, int64_t cols) {
  if (!m.p) return gtp::fail(GTP_E_ARG, "null %s", m.name);
  if (!aligned(m.p, size_of(m.dt))) return gtp::fail(GTP_E_ALIGN, "%s must be aligned to its elements", m.name);
  if (rows > 1 && m.ld < cols) return gtp::fail(GTP_E_ARG, "the row stride of %s is below cols", m.name);
  if (rows > 1 && m.ld > (int64_t(1) << 50) / rows)
    return gtp::fail(GTP_E_SHAPE, "%s spans more than 2^50 elements", m.name);
  return GTP_OK;
}

gtp::Runs runs_of(const Matrix &m, int64_t rows, int64_t cols) {
  const int64_t es = size_of(m.dt);
  return {reinterpret_cast<uintptr_t>(m.p), cols * es, {{(rows > 1 ? m.ld : cols) * es, rows}, {0, 1}, {0, 1}}};
}

gtp::Runs runs_of(const void *p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), bytes, {{bytes, 1}, {0, 1}, {0, 1}}}; }

// Whether `out` may be written where `in` is read by the thread that writes it: the same elements.
bool same_place(const Matrix &out, const Matrix &in, int64_t rows) {
  return out.p == in.p && out.dt == in.dt && (rows == 1 || out.ld == in.ld);
}

// Whether every row starts on eight elements' own size.
bool vector_rows(const Matrix &m, int64_t rows) {
  return aligned(m.p, 8 * size_of(m.dt)) && (rows == 1 || m.ld % 8 == 0);
}

}  // namespace
