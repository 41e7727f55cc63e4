// checks.h - pointer checks of the C entry points: alignment and overlap of the buffers of a call.
#pragma once

#include <cstdint>

namespace sta {

struct Range {
  const void* p;
  int64_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// Whether any of the first n_out ranges overlaps another one.
inline bool any_overlap(const Range* r, int n_out, int n) {
  for (int i = 0; i < n_out; ++i)
    for (int j = 0; j < n; ++j)
      if (j != i && overlap(r[i], r[j])) return true;
  return false;
}

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace sta
