// kda_checks.h -- argument checks shared by the host sides of libkda's entry
// points (internal; not installed).
#pragma once
#include <stdint.h>

namespace kda {

constexpr int64_t kInt32Max = 2147483647LL;

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
  bool empty() const { return lo == hi; }
};

inline Range range_of(const void* p, uint64_t bytes) {
  Range r;
  if (p && bytes) {
    r.lo = reinterpret_cast<uintptr_t>(p);
    r.hi = r.lo + bytes;
  }
  return r;
}

inline bool overlaps(const Range& a, const Range& b) {
  return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}
inline bool exact(const Range& a, const Range& b) { return !a.empty() && a.lo == b.lo && a.hi == b.hi; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace kda
