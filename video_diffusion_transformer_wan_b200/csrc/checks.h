// Argument checks of the packed-document entry points.
#pragma once
#include "internal.h"

#define WAN_REQUIRE(cond, code) \
  do {                          \
    if (!(cond)) return (code); \
  } while (0)
#define WAN_TRY(expr)              \
  do {                             \
    int _st = (expr);              \
    if (_st != WAN_OK) return _st; \
  } while (0)

namespace wan {

// An array of n rows (or entries): required, 16-byte aligned; of none: may be NULL.
inline int check_array(const void* p, int64_t n) { return n > 0 ? check_ptr(p) : check_opt_ptr(p); }

// int32 arrays are read one by one (a slice of a longer array will do): 4-byte aligned.
inline int check_ints(const int32_t* p, int64_t n) {
  if (!p) return n > 0 ? WAN_ERR_NULL : WAN_OK;
  return (reinterpret_cast<uintptr_t>(p) & 3u) == 0 ? WAN_OK : WAN_ERR_ALIGN;
}

// Rows of at least `width` elements. `whole16`: every row starts on a 16-byte boundary.
inline int check_view(const wan_rows* v, int rows, int64_t width, int dtype, bool whole16) {
  WAN_REQUIRE(v, WAN_ERR_NULL);
  WAN_TRY(check_array(v->ptr, rows));
  WAN_REQUIRE(v->row_stride >= width, WAN_ERR_SHAPE);
  if (whole16) WAN_REQUIRE(v->row_stride % (dtype == WAN_BF16 ? 8 : 4) == 0, WAN_ERR_ALIGN);
  return WAN_OK;
}

}  // namespace wan
