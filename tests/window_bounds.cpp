// Prints the bytes that the window attention's loads may touch, for each
// "left most ld D" on standard input.
#include <cstdio>

#include "engram_window_bounds.h"

int main() {
  long long left, most, ld, d;
  while (std::scanf("%lld %lld %lld %lld", &left, &most, &ld, &d) == 4)
    std::printf("%u\n", (unsigned)engram::readable_bytes((int)left, (int)most, ld, (int)d));
  return 0;
}
