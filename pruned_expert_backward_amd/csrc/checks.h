// Argument checks of the forward-side entry points (all on the host, before any
// launch).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lrmoe.h"

namespace lrmoe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Pointer rules: a NULL pointer is accepted only for an empty array.
inline lrmoe_status need(const void* p, int64_t elems) {
  if (elems == 0) return LRMOE_OK;
  if (p == nullptr) return LRMOE_ERR_NULL;
  if (!aligned16(p)) return LRMOE_ERR_ALIGN;
  return LRMOE_OK;
}

inline lrmoe_status optional(const void* p) {
  if (p != nullptr && !aligned16(p)) return LRMOE_ERR_ALIGN;
  return LRMOE_OK;
}

#define LRMOE_TRY(x)                      \
  do {                                    \
    lrmoe_status _s = (x);                \
    if (_s != LRMOE_OK) return _s;        \
  } while (0)

inline lrmoe_status hip_status(hipError_t e) {
  return e == hipSuccess ? LRMOE_OK : LRMOE_ERR_HIP;
}

}  // namespace lrmoe
