// checks.hpp -- host-side argument checks shared by the C ABI's entry points.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace moelora {

inline bool aligned(const void* p, uintptr_t to) { return p != nullptr && ((uintptr_t)p & (to - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

struct Range {
  uintptr_t lo, hi;
};
inline Range rng(const void* p, size_t bytes) { return Range{(uintptr_t)p, (uintptr_t)p + (p != nullptr ? bytes : 0)}; }
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace moelora
