// Argument checks shared by the C-ABI entry points (host code).
#pragma once

#include "common.h"

namespace lcm {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline lc_moe_status check_shape(const lc_moe_shape* s) {
  if (!s) return LC_MOE_E_NULLPTR;
  if (s->dtype != LC_MOE_F32 && s->dtype != LC_MOE_BF16) return LC_MOE_E_DTYPE;
  if (s->T < 1 || s->d < 1 || s->N < 1 || s->K < 1 || s->I < 1 || s->Z < 0) return LC_MOE_E_SHAPE;
  const long long E = static_cast<long long>(s->N) + s->Z;
  if (s->K > E || E > kMaxE || s->N > kMaxN) return LC_MOE_E_SHAPE;
  if (static_cast<long long>(s->T) * s->K >= (1LL << 31)) return LC_MOE_E_SHAPE;
  const int vec = s->dtype == LC_MOE_BF16 ? 8 : 4;
  if (s->d % vec != 0 || s->I % vec != 0) return LC_MOE_E_SHAPE;
  if (!grids_fit(*s)) return LC_MOE_E_SHAPE;
  return LC_MOE_OK;
}

// Non-null and 16-byte aligned (optional pointers may be null).
inline lc_moe_status check_ptr(const void* p, bool optional = false) {
  if (!p) return optional ? LC_MOE_OK : LC_MOE_E_NULLPTR;
  return aligned16(p) ? LC_MOE_OK : LC_MOE_E_ALIGN;
}

#define LCM_CHECK(expr)                        \
  do {                                         \
    lc_moe_status _st = (expr);                \
    if (_st != LC_MOE_OK) return _st;          \
  } while (0)
#define LCM_LAUNCH(expr)                       \
  do {                                         \
    if ((expr) != hipSuccess) return LC_MOE_E_DEVICE; \
  } while (0)

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

}  // namespace lcm
