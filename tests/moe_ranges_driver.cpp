// The weights of the experts' ranges of k, as constant expressions: one that
// overflowed would not compile.
#include <cstdint>
#include <cstdio>

#include "moe_ranges.h"

using namespace ovl;

constexpr int32_t least(int32_t items, int32_t steps, int32_t most) {
  int32_t best = INT32_MAX;
  for (int32_t r = 1; r <= kMoeMostRanges; ++r) {
    const int32_t w = moe_range_weight(items, steps, most, r);
    if (w < best) best = w;
  }
  return moe_weight_ranges(best);
}

// Ranges that are refused weigh INT32_MAX, by their number or for an empty one.
static_assert(moe_range_weight(64, 32, 4, 5) == INT32_MAX);
static_assert(moe_range_weight(64, 4, 16, 3) == INT32_MAX);
static_assert(moe_range_weight(64, 4, 16, 4) != INT32_MAX);
// No expert of this rank: nothing to cut.
static_assert(least(0, 128, 16) == 1);
// One step cannot be cut; one item of many steps is; more items than workgroups are not.
static_assert(least(1, 1, 16) == 1);
static_assert(least(1, 128, 16) == 16);
static_assert(least(4096, 32, 16) == 1);
// The largest calls: 256 experts of 2^16 x 2^13 codes (32 columns, 128 codes a step), and the other way round.
constexpr int32_t kWide = moe_range_weight(256 * 2048, 64, 16, 16), kLong = moe_range_weight(256 * 256, 512, 16, 16);
static_assert(kWide > 0 && kWide < (1 << 27) && kLong > 0 && kLong < (1 << 27));
static_assert(moe_range_weight(256 * 2048, 64, 16, 1) > 0 && moe_range_weight(256 * 256, 512, 16, 1) > 0);

int main() {
  std::printf("moe ranges ok\n");
  return 0;
}
