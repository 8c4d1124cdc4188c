// Host-side argument checks shared by the C-ABI translation units.
#pragma once

#include <stdint.h>

#include "ers.h"

namespace ers {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline ers_status check_ptr(const void* p, bool required) {
  if (p == nullptr) return required ? ERS_EINVAL : ERS_OK;
  return aligned16(p) ? ERS_OK : ERS_EPTR;
}

}  // namespace ers

#define ERS_TRY(expr)                  \
  do {                                 \
    const ers_status st_ = (expr);     \
    if (st_ != ERS_OK) return st_;     \
  } while (0)
