// Argument checks shared by the entry points of the C ABI (host code).
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

namespace ssd {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline size_t io_size(int32_t dt) { return dt == SSD_BF16 ? 2 : 4; }

// Checked product of non-negative int64 values; false on overflow.
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)bytes};
}

inline bool overlap(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline bool limits_ok(float lo, float hi) { return !isnan(lo) && !isnan(hi) && lo <= hi; }

}  // namespace ssd
