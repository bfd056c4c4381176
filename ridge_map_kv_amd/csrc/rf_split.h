// How long axes are split over workgroups: plain arithmetic, the same on the host and the device.
#pragma once

#include <stdint.h>

namespace rf {

constexpr int kSplitTries = 6;
constexpr int kMostGrains = 1 << 24;    // of one sequence: 2^30 rows in grains of 64

// Parts wanted of all sequences, where each takes `per_part` workgroups: as many as fit into `want`
// workgroups, since one too many costs a round of its own.
constexpr int parts_goal(int want, int per_part) { return want / per_part > 1 ? want / per_part : 1; }

// Least rows of a part of up to 16 query rows, where a workgroup takes `heads` key heads and a part `per_part`
// workgroups.  Parts that are joined in any case (beside prefixes, where sequences are short) have 512 rows to a workgroup,
// not 256, unless that makes less than a quarter of the workgroups wanted: with a prefix of 8,192 rows, 32 query and 8
// key heads of 128 in bf16, 1, 4 and 16 sequences of 2,048 rows take 21.6, 23.8 and 64 us with 256, 24.0, 24.9 and 61
// with 512; in fp8 4 of 512 rows 22.6 and 23.6, 8 of 2,048 37.5 and 34.9.
constexpr int least_rows(int batch, int max_len, int per_part, int want, int heads, bool joined) {
  const int many = 512 / heads;
  const int64_t workgroups = (int64_t)batch * ((max_len + many - 1) / many) * per_part;
  return joined && 4 * workgroups >= want ? many : 256 / heads;
}

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

// Groups of sequences that share prefixes.  Query rows of a block: few to a prefix stay in registers, unless one
// prefix could have many of them, since each block of 16 reads its rows again.  `all`: the batch's query rows, `mean`:
// a group's.
constexpr int prefix_block(int64_t mean, int64_t all) { return mean <= 16 && all <= 64 ? 16 : mean <= 128 ? 128 : 256; }
constexpr int query_blocks(int n, int group, int rows) { return (n * group + rows - 1) / rows; }

// Whether sequences from .. to - 1, with queries first .. end - 1, can be a group whose prefix has `len` rows; no more
// queries than its sequences may have, so that its query rows stay below 2^26.
constexpr bool is_group(int from, int to, int len, int first, int end, int batch, int max_len, int max_q, int64_t n_q) {
  return from >= 0 && to >= from && to <= batch && len >= 0 && len <= max_len && first >= 0 && end >= first &&
         end <= n_q && (int64_t)end - first <= (int64_t)(to - from) * max_q;
}
// A group counts if it also begins where those before it (of which is_group holds) have ended, in sequences and in
// queries: no sequence and no query is in two of them, so that all have at most as many blocks and pairs of a block
// and a part as the two functions below say, whatever the lists hold.
struct GroupLine {
  int seq, query;
};
constexpr bool begins_at(int from, int first, GroupLine line) { return from >= line.seq && first >= line.query; }

// `all` query rows of at most `groups` groups with queries; each group's last block may not be full.
constexpr int64_t most_blocks(int64_t all, int64_t groups, int rows) { return all / rows + groups; }
// `parts`: of one block, at most.
constexpr int64_t most_pairs(int64_t blocks, int64_t parts, int goal) {
  const int64_t pairs = blocks > goal ? blocks : goal;
  return blocks == 0 ? 1 : blocks * parts < pairs ? blocks * parts : pairs;
}
// Grains of a part of groups whose `blocks` blocks have `total` grains together.
template <typename Count>
constexpr int group_grains(int64_t total, int blocks, int goal, int least, Count parts_of) {
  return blocks < goal ? part_grains(total, blocks, goal, least, parts_of) : kMostGrains;
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
