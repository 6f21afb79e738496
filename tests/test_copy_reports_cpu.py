"""The bookkeeping by which a load warp of the wide paged attention reports its
tiles full (csrc/copy_reports.h), run on the host: every item brought in by
asynchronous copies is reported exactly once, and never before its copies have
landed, whatever run of TMA boxes came before it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_beam_shared_b200", "csrc")

# The issue loop of the load warps: per token tile an item of K and one of V,
# by boxes or by copies; a commit after every item; before an item now and then
# a wait for everything (a stage that is not free yet); after an item a wait for
# all but the last two groups.
SOURCE = r"""
#include "copy_reports.h"
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

static int run(const std::vector<int> &boxes, unsigned seed) {
  onela::CopyReports rep;
  const uint32_t items = 2 * (uint32_t)boxes.size();
  std::vector<int> reported(items, 0);
  uint32_t landed = 0, it = 0;  // copies of items below `landed` have landed
  int bad = 0;
  auto tell = [&](uint32_t upto) {
    if (!rep.due(upto)) return;
    rep.landed(upto, [&](uint32_t i) {
      if (i >= landed || i >= items || boxes[i / 2]) ++bad;
      else ++reported[i];
    });
  };
  srand(seed);
  for (uint32_t t = 0; t < boxes.size(); ++t)
    for (int kv = 0; kv < 2; ++kv, ++it) {
      if (seed && rand() % 3 == 0 && rep.pend) {
        landed = it;
        tell(it);
      }
      if (!boxes[t]) rep.mark(it);
      if (rep.pend && it >= 2) {
        landed = it - 1;
        tell(it - 1);
      }
    }
  landed = it;
  tell(it);
  for (uint32_t i = 0; i < items; ++i) bad += reported[i] != !boxes[i / 2];
  return bad;
}

int main() {
  long runs = 0, bad = 0;
  for (int before = 0; before < 200; ++before)      // box tiles before the first of copies
    for (int copies = 1; copies <= 3; ++copies)
      for (int after = 0; after < 40; after += 13)   // and box tiles behind it, then one more
        for (unsigned seed = 0; seed < 3; ++seed) {
          std::vector<int> b(before, 1);
          b.insert(b.end(), copies, 0);
          b.insert(b.end(), after, 1);
          b.push_back(0);
          ++runs;
          bad += run(b, seed) != 0;
        }
  for (unsigned seed = 1; seed < 3000; ++seed) {     // any mixture
    srand(seed);
    std::vector<int> b(1 + rand() % 150);
    const int share = 1 + rand() % 50;
    for (int &x : b) x = rand() % share != 0;
    ++runs;
    bad += run(b, seed % 2 ? seed : 0) != 0;
  }
  printf("%ld %ld\n", runs, bad);
}
"""


def test_items_are_reported_once_and_not_before_they_landed(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "reports.cpp", tmp_path / "reports"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    runs, bad = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert runs > 5000 and bad == 0
