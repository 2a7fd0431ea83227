// The join of the gradient norm's sums: a foreign verdict reaches the total
// from any place, through two levels, beside finite, infinite and NaN sums.
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include "clip_sum.h"

using ovl::ClipTotal;
using ovl::kClipForeign;

int main() {
  int failures = 0;
  const double inf = HUGE_VAL, nan = std::nan("");
  for (double other : {0.0, 2.5, 1e300, inf, nan})
    for (int at = -1; at < 16; ++at) {  // -1: no foreign term
      ClipTotal total;
      double plain = 0;
      for (int g = 0; g < 4; ++g) {
        ClipTotal group;
        for (int w = 0; w < 4; ++w) {
          const double v = (g + w) % 2 ? other : 1.0;
          group.add(4 * g + w == at ? kClipForeign : v);
          plain += v;
        }
        total.add(group.word());
      }
      if (total.foreign != (at >= 0)) ++failures;
      if (at < 0 && !(total.sum == plain || (std::isnan(total.sum) && std::isnan(plain)))) ++failures;
    }
  std::printf(failures ? "%d failures\n" : "clip sum ok\n", failures);
  return failures != 0;
}
