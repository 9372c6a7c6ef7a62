// Prints for every "layout rows k units" line of the input (layout 0 rows, 1
// mixed, 2 columns) how such a product runs: tile, splits of k, and whether its
// lines begin at any element or are copied first.
#include <cstdio>

#include "ops_kernels.h"

int main() {
  const char* names[] = {"direct", "few", "mid", "wide", "tall", "big"};
  int layout, units;
  long long rows, k;
  while (std::scanf("%d %lld %lld %d", &layout, &rows, &k, &units) == 4) {
    const bool any = (layout == twell::LINEAR_ROWS ? k : units) % 8 != 0;
    const twell::LinearPlan p = twell::linear_plan((twell::LinearLayout)layout, rows, k, units, any);
    std::printf("%s %s %s\n", names[p.tile], p.splits > 1 ? "split" : "whole", p.pad ? "copied" : any ? "any" : "aligned");
  }
  return 0;
}
