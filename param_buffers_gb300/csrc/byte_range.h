// The bytes an argument spans, for the checks that outputs share none with inputs or each other.
#pragma once
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

}  // namespace gtp
