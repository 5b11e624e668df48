// engram_linear_plan.h -- how the linear layer's products are cut into
// workgroups (internal; host arithmetic only).
#pragma once

#include <stdint.h>

namespace engram {

constexpr int kBk = 64;  // contraction values of a stage

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a product is cut into workgroups.  Tiles are 256 x 256, one to a CU, or
// 128 x 128, two to a CU with two stages each or one with four: where fewer
// tiles than two to a CU are to be had, the deeper one keeps as much on its way
// (128 x 2560 x 25600: 28 us against 36).  Few rows take 64 x 128 or 32 x 128,
// three or four to a CU, whose LDS then holds more of W on its way.  Tiles that
// fill whole rounds of the chip's places are made whole; those of the last,
// partial round may be cut along the contraction, into parts of at least four
// stages (4000 x 5120 x 5120: 202 us against 234 uncut; 4096 x 25600 x 2560, 160
// tiles of 256^2 in three parts: 557 against 612).
// The cheapest by the costs below is taken, which were fitted to all three
// shapes over fourteen sizes (256^2, 128^2 and 128^2 deep, us: 4000 x 5120 x 5120
// 197, 208, 247; 2048 x 5120 x 5120 126, 110, 133; 1000 x 1368 x 5120 41, 27, 34;
// 2000 x 640 x 6000 24, 35, 32; 700 x 700 x 700 21, 12, 13).
struct Shape {
  int i, j, places;
  double stage, round;  // microseconds of a stage with all places taken, and of a round besides its stages
};
constexpr Shape kShapes[] = {{256, 256, 256, 1.55, 8.0},
                             {128, 128, 512, 1.00, 3.0},
                             {128, 128, 256, 0.60, 6.0},
                             {64, 128, 768, 0.80, 2.0},
                             {32, 128, 1024, 0.80, 2.0}};

constexpr int64_t kMostFill = 3;

struct Plan {
  int shape;
  int ti, tj, whole, cut, parts;
  int64_t c_part;
  double cost;
};

inline Plan plan_with(int shape, int64_t I, int64_t J, int64_t C) {
  Plan p{};
  p.shape = shape;
  const Shape& s = kShapes[shape];
  p.ti = (int)up(I, s.i);
  p.tj = (int)up(J, s.j);
  const int64_t tiles = (int64_t)p.ti * p.tj, stages = up(C, kBk);
  const int64_t last = tiles % s.places;
  // microseconds: full rounds, then the last tiles in as many parts as is cheapest; cut tiles' sums
  // are written and read again by a second launch
  const double whole = (double)(tiles / s.places) * (s.stage * stages + s.round);
  for (int64_t fill = 0; fill <= kMostFill; ++fill) {
    int64_t n = fill && last ? fill * s.places / last : 1;  // not cut, or to fill one, two, ... rounds
    if (n > stages / 4) n = stages / 4;
    if (n < 1) n = 1;
    const int64_t part_stages = up(stages, n), parts = up(stages, part_stages);
    const double rounds = (double)up(last * parts, s.places), bytes = (double)(last * parts) * s.i * s.j * 8.0;
    const double cost = whole + rounds * s.stage * part_stages + (parts > 1 ? 8.0 + bytes / 4.0e6 : rounds * s.round);
    if (fill && cost >= p.cost) continue;
    p.cost = cost;
    p.parts = (int)parts;
    p.c_part = part_stages * kBk;
    p.cut = parts > 1 ? (int)last : 0;
  }
  p.whole = (int)tiles - p.cut;
  return p;
}

inline Plan plan_of(int64_t I, int64_t J, int64_t C) {
  if (I <= 32) return plan_with(4, I, J, C);
  if (I <= 64) return plan_with(3, I, J, C);
  Plan best = plan_with(0, I, J, C);
  for (int shape = 1; shape <= 2; ++shape) {
    const Plan p = plan_with(shape, I, J, C);
    if (p.cost < best.cost) best = p;
  }
  return best;
}

// The forward's calls that take no tiles: a few rows of x, up to kVectorRows of
// them with plain products, and up to kFewRows at a small W straight from
// memory into the matrix cores.
constexpr int64_t kVectorRows = 4;
constexpr int64_t kFewRows = 16, kSmallWeight = 1 << 24;  // rows, and values of W, of rows_kernel
inline bool few_rows(int64_t N, int64_t K, int64_t M) { return N <= kVectorRows || (N <= kFewRows && K * M <= kSmallWeight); }

}  // namespace engram
