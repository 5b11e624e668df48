// Prints how the linear layer cuts products into workgroups: for each "I J C" on
// standard input the tile shape, whole and cut tiles and parts of a cut one, and
// whether a forward of I rows, C values and J outputs takes no tiles.
#include <cstdio>

#include "engram_linear_plan.h"

int main() {
  long long i, j, c;
  while (std::scanf("%lld %lld %lld", &i, &j, &c) == 3) {
    const engram::Plan p = engram::plan_of(i, j, c);
    std::printf("%d %d %d %d %d\n", p.shape, p.whole, p.cut, p.cut ? p.parts : 1, (int)engram::few_rows(i, c, j));
  }
  return 0;
}
