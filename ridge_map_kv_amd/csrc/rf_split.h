// How long axes are split over workgroups: plain arithmetic, the same on the host and the device.
#pragma once

#include <stdint.h>

namespace rf {

constexpr int kSplitTries = 6;
constexpr int kMostGrains = 1 << 24;    // of one sequence: 2^30 rows in grains of 64

// Parts wanted of all sequences, where each takes `per_part` workgroups: as many as fit into `want`
// workgroups, since one too many costs a round of its own.
constexpr int parts_goal(int want, int per_part) { return want / per_part > 1 ? want / per_part : 1; }

// Grains of one part where sequences of together `total` grains, cut into parts each of its own, come to
// `goal` parts at most; goal > batch, and `least` grains are taken at least.  parts_of(each) counts the
// parts for a size; it never rises with the size.  The smallest that might do is total / goal, and
// total / (goal - batch) does, since parts_of(each) <= total / each + batch: between them by halves, a
// few times (the rest is then 1/64 of the difference).
template <typename Count>
constexpr int part_grains(int64_t total, int batch, int goal, int least, Count parts_of) {
  const auto size = [&](int64_t parts) {
    const int64_t each = (total + parts - 1) / parts;
    return (int)(each < least ? least : each > kMostGrains ? kMostGrains : each);
  };
  int lo = size(goal), hi = size(goal - batch);
  if (lo >= hi || parts_of(lo) <= goal) return lo;
  ++lo;
  for (int i = 0; i < kSplitTries && lo < hi; ++i) {
    const int mid = lo + (hi - lo) / 2;
    if (parts_of(mid) <= goal)
      hi = mid;
    else
      lo = mid + 1;
  }
  return hi;
}

// Rows of a workgroup where `units` axes of `rows` rows are split over workgroups that each want a
// compute unit (of kUnitsOfChip), in multiples of `step` rows: as many as fit into one round or, if those of
// a second round are so much shorter that both are over sooner, as many as leave no compute unit out.
constexpr int kUnitsOfChip = 256;
constexpr int chunk_rows(int64_t units, int rows, int step) {
  const auto chunk = [&](int64_t splits) {
    const int64_t each = splits > 1 ? (rows + splits - 1) / splits : rows;
    return (each + step - 1) / step * step;
  };
  const auto time = [&](int64_t each) {
    return (units * ((rows + each - 1) / each) + kUnitsOfChip - 1) / kUnitsOfChip * each;
  };
  const int64_t few = chunk(kUnitsOfChip / units), many = chunk((kUnitsOfChip + units - 1) / units);
  return (int)(time(many) < time(few) ? many : few);
}

}  // namespace rf
