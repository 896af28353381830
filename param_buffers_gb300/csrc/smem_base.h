// Where a block's dynamic shared memory starts: behind the bytes that the system keeps for itself and the kernel's own
// static shared memory.  A kernel that fills the whole of it cannot afford to align it a second time.
#pragma once
#include <cstddef>

#include "status.h"

namespace gtp {

// GTP_OK where dynamic shared memory starts on a multiple of `align` bytes, given what lies before it.
inline gtp_status check_dynamic_base(const char *what, size_t reserved_bytes, size_t static_bytes, size_t align) {
  if (reserved_bytes % align == 0 && static_bytes % align == 0) return GTP_OK;
  return fail(GTP_E_CUDA, "%s: dynamic shared memory behind %zu reserved and %zu static bytes is not on %zu", what,
              reserved_bytes, static_bytes, align);
}

}  // namespace gtp
