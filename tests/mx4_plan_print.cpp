// Prints for every "tokens columns units" line of the input how linear_mx4 and
// matmul_mx4 of that size run: the plan of each and the direct product's tile.
#include <cstdio>

#include "ops_kernels.h"

int main() {
  const char* names[] = {"fused", "direct", "mid", "big"};
  long long n;
  int cols, units;
  while (std::scanf("%lld %d %d", &n, &cols, &units) == 3)
    std::printf("%s %s %d\n", names[twell::mx4_plan(n, cols, units, false)],
                names[twell::mx4_plan(n, cols, units, true)], twell::mx4_direct_tile(n, cols, units));
  return 0;
}
