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
