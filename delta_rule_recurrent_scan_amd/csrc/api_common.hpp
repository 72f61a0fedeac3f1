// Host-side argument checks shared by the C ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/osdn.h"

namespace osdn_api {

inline bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
inline bool dtype_ok(int t) { return t == OSDN_F32 || t == OSDN_BF16; }
inline size_t elem(int dtype) { return dtype == OSDN_BF16 ? 2 : 4; }
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
  bool valid() const { return lo != 0 && hi > lo; }
};
inline Range rng(const void* p, size_t bytes) {
  return Range{(uintptr_t)p, (uintptr_t)p + (p ? bytes : 0)};
}
inline bool overlap(Range a, Range b) {
  return a.valid() && b.valid() && a.lo < b.hi && b.lo < a.hi;
}
inline bool same(Range a, Range b) { return a.lo == b.lo && a.hi == b.hi; }

// Outputs must not overlap inputs or each other, except for the exact
// in-place pairs listed in `allowed` (output index, input index).
template <int NO, int NI>
bool aliasing_ok(const Range (&outs)[NO], const Range (&ins)[NI], const int (*allowed)[2],
                 int nallowed) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j) {
      if (!overlap(outs[i], ins[j])) continue;
      bool ok = false;
      for (int a = 0; a < nallowed; ++a)
        if (allowed[a][0] == i && allowed[a][1] == j && same(outs[i], ins[j])) ok = true;
      if (!ok) return false;
    }
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return false;
  }
  return true;
}

}  // namespace osdn_api
