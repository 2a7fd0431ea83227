// What cutting the experts' items into ranges of k costs.
#pragma once

#include <stdint.h>

namespace ovl {

constexpr int kMoeGroups = 256;    // workgroups of the experts' launches: one a compute unit
constexpr int kMoeMostRanges = 16;

// Rounds of kMoeGroups items times the steps of one, an item counting a fixed
// part beside its steps (about six steps of start and reduction; four more
// where the ranges' sums meet in memory).  Sixteen times that and the ranges
// less one, so that the least of several names its ranges in its low bits;
// INT32_MAX where they are more than `most` or leave one empty.  An expert's
// matrix has at most 2^30 codes, an item 32 x 128 of them a step: with 256
// experts the cost stays below 2^23 and the word below 2^27.
constexpr int32_t moe_range_weight(int32_t items, int32_t steps, int32_t most, int32_t ranges) {
  const int32_t per = (steps + ranges - 1) / ranges;
  if (ranges > most || (ranges - 1) * per >= steps) return INT32_MAX;
  const int32_t rounds = (items * ranges + kMoeGroups - 1) / kMoeGroups;
  return rounds * (per + (ranges > 1 ? 10 : 6)) * kMoeMostRanges + ranges - 1;
}
constexpr int32_t moe_weight_ranges(int32_t weight) {
  return weight == INT32_MAX ? 1 : weight % kMoeMostRanges + 1;
}

}  // namespace ovl
