// Argument checks of the entry points beside the pruned backward (all on the host,
// before any launch).
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

constexpr int64_t kMaxRows = int64_t(1) << 31;

inline lrmoe_status check_dtype(int32_t dtype) {
  return dtype == LRMOE_F32 || dtype == LRMOE_BF16 ? LRMOE_OK : LRMOE_ERR_DTYPE;
}

// A row length: 1 .. 2^20, whole 16-byte pieces in the storage type.
inline lrmoe_status check_width(int32_t dtype, int64_t d) {
  if (d < 1 || d > (1 << 20)) return LRMOE_ERR_SHAPE;
  return d % (dtype == LRMOE_BF16 ? 8 : 4) == 0 ? LRMOE_OK : LRMOE_ERR_ALIGN;
}

inline lrmoe_status check_experts(int32_t E) {
  return E >= 1 && E <= LRMOE_MAX_EXPERTS ? LRMOE_OK : LRMOE_ERR_INVALID;
}

inline lrmoe_status check_act(int32_t act) {
  return act >= LRMOE_ACT_NONE && act <= LRMOE_ACT_SWIGLU ? LRMOE_OK : LRMOE_ERR_INVALID;
}

inline lrmoe_status check_forward(const lrmoe_forward* fw) {
  if (fw == nullptr) return LRMOE_ERR_NULL;
  LRMOE_TRY(check_experts(fw->E));
  LRMOE_TRY(check_act(fw->act));
  LRMOE_TRY(check_dtype(fw->dtype));
  if (fw->P < 0 || fw->P >= kMaxRows || fw->T < 0 || fw->T >= kMaxRows) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(check_width(fw->dtype, fw->d_in));
  if (fw->act == LRMOE_ACT_SWIGLU) {
    if (fw->d_out % 2 != 0) return LRMOE_ERR_ALIGN;
    return check_width(fw->dtype, fw->d_out / 2);
  }
  return check_width(fw->dtype, fw->d_out);
}

inline hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace lrmoe
