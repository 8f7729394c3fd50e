// gs_args.h -- the argument checks the C entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gsfp8.h"

namespace gs {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}

inline size_t dtype_size(int dt) { return dt == GS_F32 ? 4 : 2; }
inline bool valid_dtype(int dt) { return dt == GS_F16 || dt == GS_BF16 || dt == GS_F32; }
inline bool valid_fmt(int f) { return f == GS_E4M3 || f == GS_E5M2; }

inline bool mul_ok(int64_t a, int64_t b) {
  return a >= 0 && b >= 0 && (b == 0 || a <= INT64_MAX / b);
}

}  // namespace gs
