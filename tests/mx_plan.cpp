/* Prints the kernel that each product takes: lines of rows of a, rows of b, columns,
 * format of a, of b, 1 for an fp32 result in; strips a side of the few-row kernel (0:
 * the many-row kernel), 64-result units a side of that one, splits out. */
#include <cstdio>

#include "nc_mx_plan.h"

int main() {
  long long m, n, k;
  int fa, fb, f32;
  while (std::scanf("%lld %lld %lld %d %d %d", &m, &n, &k, &fa, &fb, &f32) == 6) {
    const nc::MxPlan p = nc::plan_of(m, n, (k + 255) / 256, fa, fb, f32 != 0);
    std::printf("%d %d %d\n", p.t, p.w, (int)p.splits);
  }
  return 0;
}
