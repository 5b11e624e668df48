// engram_window_bounds.h -- how far a load of the window attention's tiles may read
// (internal; host code can include it).
#pragma once

#include <stdint.h>

namespace engram {

// Bytes from the first of `left` rows on (ld values apart, the first D of each
// wanted) that loads of up to `most` rows may touch: to the end of the last row
// that is there.  `left` may be all that is left of a sequence; only `most` rows of
// it count, so that the product does not pass 32 bits, and what a load names
// beyond the bound (kBeyond, for one) stays beyond it: 128 rows of
// ENGRAM_LD_MAX = 2^20 values are 2^28 bytes.
constexpr uint32_t readable_bytes(int left, int most, int64_t ld, int D) {
  const int rows = left < most ? left : most;
  return rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)(ld * 2) + (uint32_t)(D * 2) : 0u;
}

}  // namespace engram
