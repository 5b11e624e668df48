// engram_sequences.h -- the sequences that a cu_seqlens array cuts the tokens
// into, as kernels look them up (gfx950, internal).
#pragma once

#include "engram_device.h"

namespace engram {

// The array is the caller's and lies in device memory: bounds are clamped to the
// tokens there are, so that no content of it leads out of the arrays.  Everything
// here is the same in all lanes of a wave.
struct Sequences {
  const int64_t* cu;  // [B + 1]
  int64_t N;
  int B;
  __device__ __forceinline__ int64_t bound(int i) const {
    int64_t v = cu[i];
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const int32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    v = (int64_t)(((uint64_t)(uint32_t)hi << 32) | lo);
    return v < 0 ? 0 : (v > N ? N : v);
  }
  __device__ __forceinline__ int64_t start(int i) const { return bound(i); }
  __device__ __forceinline__ int64_t end(int i) const { return bound(i + 1); }
  // The last sequence whose key(its start, its number) is at most `most`, for keys
  // that rise with the number (0 if none is), and its bounds: sixty-four starts at
  // a time, one load for up to 63 sequences.
  // `asked`: the first of these loads, which may so be on its way before others are.
  __device__ __forceinline__ int64_t ask() const {
    const int i = (int)(threadIdx.x & 63) * ((B + 63) / 64);
    return cu[i <= B ? i : B];
  }
  template <typename F>
  __device__ __forceinline__ int last_at_most(int64_t most, F key, int64_t* start, int64_t* end) const {
    return last_at_most(most, key, start, end, ask());
  }
  template <typename F>
  __device__ __forceinline__ int last_at_most(int64_t most, F key, int64_t* start, int64_t* end, int64_t asked) const {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = B;
    for (int64_t raw = asked;; raw = cu[lo + lane * ((n + 63) / 64) <= B ? lo + lane * ((n + 63) / 64) : B]) {
      const int step = (n + 63) / 64, i = lo + lane * step;
      const int64_t at = raw < 0 ? 0 : (raw > N ? N : raw);
      const uint64_t in = __ballot(lane * step < n && key(at, i) <= most);
      const int last = in ? 63 - __builtin_clzll(in) : 0;
      if (step == 1) {
        if (n < 64) {
          *start = from_lane(at, last);
          *end = from_lane(at, last + 1);
        } else {
          *start = bound(lo + last);
          *end = bound(lo + last + 1);
        }
        return lo + last;
      }
      n = n - last * step < step ? n - last * step : step;
      lo += last * step;
    }
  }
  static __device__ __forceinline__ int64_t from_lane(int64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
  }
};

}  // namespace engram
