// Prints the launch plans of the RMS norms for "rows cols es vec shift pair"
// lines: form vpt x y of the norm, then form vpt x y full slot stages parts of
// the gradients with ds and dw.
#include <cstdio>

#include "norm_plan.h"

int main() {
  long long rows, cols;
  int es, vec, shift, pair;
  while (std::scanf("%lld %lld %d %d %d %d", &rows, &cols, &es, &vec, &shift, &pair) == 6) {
    const msb::NormReach by{vec != 0, shift != 0, pair};
    const msb::NormPlan p = msb::norm_plan(cols, es, by);
    const msb::NormBwdPlan b = msb::norm_bwd_plan(rows, cols, es, by, true, true);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d %lld\n", static_cast<int>(p.form), p.vpt, p.x, p.y,
                static_cast<int>(b.p.form), b.p.vpt, b.p.x, b.p.y, b.full ? 1 : 0, b.slot, b.stages,
                static_cast<long long>(b.parts));
  }
  return 0;
}
