"""CPU tests of how the cache calls split long caches over workgroups (rf_split.h, the same code on
the host and the device): never more parts than fit, and close to the fewest rows each."""

import os
import shutil
import subprocess

import pytest

from ridge_map_kv_amd import binding as B

CSRC = os.path.join(os.path.dirname(B.LIB_PATH), "csrc")

# random batches: reports those whose parts exceed the goal, and those with a part of more than the
# smallest size that fits and 1/32 of the range in which it is looked for
PARTS = r"""
#include "rf_split.h"
#include <random>
#include <stdio.h>
#include <vector>

int main() {
  std::mt19937_64 g(7);
  const auto below = [&](int64_t n) { return (int64_t)(g() % (uint64_t)n); };
  int over = 0, large = 0;
  for (int trial = 0; trial < 40000; ++trial) {
    const int goal = 2 + (int)below(trial % 3 ? 60 : 1023), batch = 1 + (int)below(goal - 1);
    const int least = trial % 2 ? 2 : 4;
    const int64_t longest = (int64_t)1 << below(trial % 50 ? 12 : 25);
    std::vector<int64_t> grains(batch);
    int64_t total = 0;
    for (auto& x : grains) {
      x = below(4) ? below(longest) + (longest == 1 << 24) : below(8);
      total += x;
    }
    const auto count = [&](int each) {
      int64_t parts = 0;
      for (auto x : grains) parts += (x + each - 1) / each;
      return (int)parts;
    };
    const int each = rf::part_grains(total, batch, goal, least, count);
    over += each < least || count(each) > goal;
    int fits = each;                                  // the smallest that does
    while (fits > least && fits - 1 >= (total + goal - 1) / goal && count(fits - 1) <= goal && each - fits < 4096) --fits;
    const int64_t range = (total + goal - batch - 1) / (goal - batch) - (total + goal - 1) / goal;
    large += each - fits > range / 32 + 1;
  }
  printf("%d %d\n", over, large);
  for (int per = 1; per < 2000; ++per)
    if (rf::parts_goal(256, per) * per > 256 && rf::parts_goal(256, per) > 1) return 1;
  return 0;
}
"""

# the chunk of every number of axes, and of random lengths: covers the rows in whole steps, and no more
# rounds of workgroups times rows than the two numbers of parts that it chooses from
CHUNKS = r"""
#include "rf_split.h"
#include <initializer_list>
#include <stdio.h>

int main() {
  const int step = 512;
  for (int units = 1; units < 1000; ++units)
    for (int rows = 1; rows < 70000; rows = rows * 5 / 4 + 1) {
      const int64_t each = rf::chunk_rows(units, rows, step);
      if (each < 1 || each % step) return 1;
      const auto rounds = [&](int64_t chunk) { return (units * ((rows + chunk - 1) / chunk) + 255) / 256; };
      for (int64_t s : {256 / units, (256 + units - 1) / units}) {
        if (s < 1) s = 1;
        const int64_t other = ((rows + s - 1) / s + step - 1) / step * step;
        if (rounds(each) * each > rounds(other) * other) return 2;
      }
    }
  for (int batch : {3, 5, 6, 9, 12}) printf("%d ", rf::chunk_rows(8 * batch, 32768, step));
  return 0;
}
"""

# random lists of groups and queries, in order and not: the pairs of a part and a block of query rows that the groups
# which count come to, and those for which there is room; the same without the order of the groups
GROUPS = r"""
#include "rf_split.h"
#include <algorithm>
#include <random>
#include <stdio.h>
#include <vector>

int main() {
  std::mt19937_64 g(11);
  const auto below = [&](int64_t n) { return (int64_t)(g() % (uint64_t)n); };
  int over = 0, over_unordered = 0, left_out = 0, bad = 0, twice = 0;
  for (int trial = 0; trial < 60000; ++trial) {
    const int batch = 1 + (int)below(trial % 2 ? 12 : 300), groups = 1 + (int)below(trial % 3 ? 9 : 200);
    const int max_q = 1 + (int)below(trial % 5 ? 4 : 64), group = 1 + (int)below(trial % 7 ? 8 : 512);
    const int max_len = 1 + (int)below((int64_t)1 << (trial % 50 ? 9 : 30));
    // lists in order, of any numbers, and in order but for some entries or a part that comes again
    const auto list = [&](int n, int most, int kind) {
      std::vector<int> x(n);
      for (auto& v : x) v = (int)below(most + 1);
      if (kind != 1) std::sort(x.begin(), x.end());
      if (kind == 2) for (int i = 0; i < 1 + n / 8; ++i) x[below(n)] = (int)below(most + 4) - 2;
      if (kind == 3) for (int i = 0; i + 1 < n; ++i) x[i] = i % 2 ? x[n / 2] : 0;
      return x;
    };
    const bool ordered = trial % 4 == 0;
    std::vector<int> starts = list(groups + 1, batch, ordered ? 0 : (int)below(4)), queries(batch + 1), lens(groups);
    const int kind = ordered ? 0 : (int)below(4);
    if (kind == 0) {
      for (int i = 0; i < batch; ++i) queries[i + 1] = queries[i] + (int)below(max_q + 1);
    } else {
      queries = list(batch + 1, (int)below((int64_t)batch * max_q + 1), kind);
    }
    const int64_t n_q = kind == 0 || below(2) ? *std::max_element(queries.begin(), queries.end()) : queries[batch];
    for (auto& v : lens) v = ordered || below(9) ? (int)below((int64_t)max_len + 1) : (int)below(2) - 1;
    if (n_q < 0) continue;
    // as the host lays a call out
    const int64_t most = (int64_t)batch * max_q, n = n_q < most ? n_q : most, with = n < groups ? n : groups, all = n * group;
    const int rows = rf::prefix_block(with ? all / with : 0, all), least = rows == 16 ? 64 << below(3) : 128;
    const int goal = rf::parts_goal(rows == 16 ? 1024 : 256, 1 + (int)below(64));
    const int64_t launched = rf::most_pairs(rf::most_blocks(all, with, rows), (max_len + least - 1) / least, goal);
    // as the device counts them
    struct Seen { int blocks, grains; };
    const auto numbered = [&](bool in_order, int* counted) {
      std::vector<Seen> seen;
      std::vector<char> of_query(n_q), of_seq(batch);
      rf::GroupLine line = {0, 0};
      int64_t total = 0, blocks = 0;
      *counted = 0;
      for (int i = 0; i < groups; ++i) {
        const int from = starts[i], to = starts[i + 1];
        if (from < 0 || from > batch || to < 0 || to > batch) continue;
        const int first = queries[from], end = queries[to];
        if (!rf::is_group(from, to, lens[i], first, end, batch, max_len, max_q, n_q)) continue;
        const bool counts = !in_order || rf::begins_at(from, first, line);
        line = {std::max(line.seq, to), std::max(line.query, end)};
        if (!counts) continue;
        ++*counted;
        if (in_order) {
          for (int q = first; q < end; ++q) twice += of_query[q]++ != 0;
          for (int s = from; s < to; ++s) twice += of_seq[s]++ != 0;
        }
        if (end == first || lens[i] == 0) continue;
        seen.push_back({rf::query_blocks(end - first, group, rows), (lens[i] + 63) / 64});
        total += (int64_t)seen.back().blocks * seen.back().grains;
        blocks += seen.back().blocks;
      }
      const auto parts = [&](int each) {
        int64_t x = 0;
        for (auto s : seen) x += (int64_t)s.blocks * ((s.grains + each - 1) / each);
        return x;
      };
      if (in_order) bad += blocks > 1 << 26;
      return parts(rf::group_grains(total, (int)blocks, goal, least / 64, [&](int each) { return (int)parts(each); }));
    };
    int counted, loose;
    over += numbered(true, &counted) > launched;
    over_unordered += numbered(false, &loose) > launched;
    left_out += ordered && counted != groups;
  }
  printf("%d %d %d %d %d\n", over, left_out, bad, twice, over_unordered);
  return 0;
}
"""

# least rows of a part, printed; never so few workgroups because of long parts that most of the chip is left out
LEAST = r"""
#include "rf_split.h"
#include <initializer_list>
#include <stdio.h>

int main() {
  for (int batch = 1; batch < 100; batch += batch / 8 + 1)
    for (int len = 1; len < 40000; len = len * 5 / 4 + 1)
      for (int heads : {1, 2, 4})
        for (int per_part : {1, 2, 8, 16})
          for (int want : {512, 1024}) {
            const int alone = rf::least_rows(batch, len, per_part, want, heads, false), least = rf::least_rows(batch, len, per_part, want, heads, true);
            const auto workgroups = [&](int rows) { return batch * ((len + rows - 1) / rows) * per_part; };
            if (alone != 256 / heads || (least != alone && least != 2 * alone)) return 1;
            if (least != alone && 4 * workgroups(least) < want) return 2;
          }
  const auto show = [](int batch, int len, int per_part, int want, int heads) { printf("%d ", rf::least_rows(batch, len, per_part, want, heads, true)); };
  show(64, 512, 8, 1024, 1), show(4, 2048, 8, 1024, 1), show(1, 65536, 8, 1024, 1), show(48, 2048, 2, 512, 4), show(4, 512, 2, 512, 4);
  return 0;
}
"""


def _run(tmp_path, source):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    (tmp_path / "split.cpp").write_text(source)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                    str(tmp_path / "split.cpp"), "-o", str(tmp_path / "split")], check=True)
    return subprocess.run([str(tmp_path / "split")], check=True, capture_output=True, text=True).stdout.split()


def test_parts_never_exceed_the_goal(tmp_path):
    over, large = _run(tmp_path, PARTS)
    assert int(over) == 0 and int(large) == 0


def test_groups_never_exceed_the_pairs_that_are_launched(tmp_path):
    over, left_out, bad, twice, over_unordered = (int(x) for x in _run(tmp_path, GROUPS))
    assert over == 0 and bad == 0 and twice == 0
    assert left_out == 0                                  # in lists that are in order every group counts
    assert over_unordered > 100                           # the lists would, without the order


@pytest.mark.parametrize("heads,n_kv,max_q", [(5, 5, 64), (6, 3, 64), (6, 6, 33), (80, 8, 64), (8, 8, 64), (24, 3, 20),
                                              (10, 5, 1), (12, 6, 2), (32, 8, 1)])
def test_attention_fits_one_round_of_workgroups(heads, n_kv, max_q):
    # the workspace holds one partial result a part; workgroups: parts, key heads, blocks of query rows
    hd, rows = 128, max_q * heads // n_kv
    kv = B.rf_paged_batch(1 << 20, 1 << 20, 1 << 14, 2, 1 << 18, 16, 1 << 15, n_kv, hd)
    size = B.ridgefill_tree_attention_workspace_bytes(kv, heads, max_q)
    parts = (size - 256) // (n_kv * rows * (8 + 4 * hd))
    want, block = (1024, 16) if rows <= 16 else (256, 128) if rows <= 128 else (256, 256)
    assert want * 3 // 4 < parts * n_kv * -(-rows // block) <= want


def test_weight_chunks_leave_no_stragglers(tmp_path):
    # 8 key heads, 32,768 rows: workgroups of all batches fit 256 compute units
    chunks = [int(x) for x in _run(tmp_path, CHUNKS)]
    for batch, chunk in zip((3, 5, 6, 9, 12), chunks):
        assert 8 * batch * -(-32768 // chunk) <= 256


def test_parts_beside_prefixes_are_not_too_long_for_few_sequences(tmp_path):
    assert [int(x) for x in _run(tmp_path, LEAST)] == [512, 256, 512, 128, 64]
