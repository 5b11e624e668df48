// engram_check.h -- host-side checks of pointers shared by the C entry points
// (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engram.h"

namespace engram {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + (uintptr_t)bytes};
}

inline bool overlaps(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Outputs (and scratch) may overlap neither an input nor each other.
inline bool any_overlap(const Range* in, int nin, const Range* out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i], in[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i], out[j])) return true;
  }
  return false;
}

// Rows of `width` bytes that begin `ld` bytes apart (one row: ld is not
// looked at; a null pointer is an argument that is not there).
struct Rows {
  const void* p;
  int64_t rows, ld, width;
};

inline Rows flat(const void* p, int64_t bytes) { return Rows{p, 1, 0, bytes}; }

inline Range range_of(const Rows& r) {
  return r.p ? range_of(r.p, (r.rows - 1) * r.ld + r.width) : Range{0, 0};
}

// Whether two sets of rows share a byte.  Sets whose ranges meet are apart
// only if they are different columns of the same rows (queries and keys in one
// packed row, say); sets that meet in any other way count as overlapping.
inline bool overlaps(const Rows& a, const Rows& b) {
  const Range ra = range_of(a), rb = range_of(b);
  if (!overlaps(ra, rb)) return false;
  if (a.rows > 1 && b.rows > 1 && a.ld == b.ld) {
    const int64_t ld = a.ld;
    const int64_t d = (int64_t)(rb.lo >= ra.lo ? (rb.lo - ra.lo) % (uintptr_t)ld
                                               : ((uintptr_t)ld - (ra.lo - rb.lo) % (uintptr_t)ld) % (uintptr_t)ld);
    return !(d >= a.width && d + b.width <= ld);
  }
  return true;
}

inline bool any_overlap(const Rows* in, int nin, const Rows* out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i], in[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i], out[j])) return true;
  }
  return false;
}

// The status of a launch; remembers the HIP error of the calling thread.
engram_status launched(hipError_t e);

}  // namespace engram
