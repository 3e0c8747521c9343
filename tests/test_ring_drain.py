"""The rule by which the window and paged forward awaits its last copies, on the CPU: a
simulated ring whose warps stop at any moment."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_rank_hybrid_simhash_b200", "csrc")

# Loads of a slot follow one another: load i may start once load i - slots has been read, and the
# products read in order.  At any stop, the loads that have started and have not been read may be in
# flight: each must be awaited, and only a slot's newest load may be (its barrier's parity says
# nothing of earlier ones).
PROGRAM = r"""
#include <cstdio>
#include <set>
#include <tuple>
#include <vector>
#include "ring_drain.h"
using elsaa::RingDrain;
int main() {
  long states = 0;
  for (uint32_t slots : {5u, 8u})
    for (uint32_t total = 0; total <= 13; ++total) {   // blocks: K and V of each
      std::set<std::tuple<uint32_t, uint32_t, uint32_t>> seen;
      std::vector<std::tuple<uint32_t, uint32_t, uint32_t>> todo{{0u, 0u, 0u}};
      while (!todo.empty()) {
        const auto at = todo.back();
        todo.pop_back();
        if (!seen.insert(at).second) continue;
        ++states;
        const auto [k, v, read] = at;   // loads started by K and V, loads read
        const RingDrain r{slots, k, v};
        for (uint32_t i = 0; i < 2 * total + 2 * slots; ++i) {
          const bool started = i / 2 < (i & 1 ? v : k), newer = (i + slots) / 2 < ((i + slots) & 1 ? v : k);
          const bool awaited = i >= r.begin() && i < r.end() && r.open(i);
          if (started && i >= read && !awaited) return std::printf("load %u not awaited: slots %u, k %u, v %u, read %u\n", i, slots, k, v, read), 1;
          if (awaited && (!started || newer)) return std::printf("load %u awaited: slots %u, k %u, v %u, read %u\n", i, slots, k, v, read), 1;
        }
        auto free = [&](uint32_t i) { return i < slots || i - slots < read; };
        if (k < total && free(2 * k)) todo.push_back({k + 1, v, read});
        if (v < total && free(2 * v + 1)) todo.push_back({k, v + 1, read});
        if (read / 2 < (read & 1 ? v : k)) todo.push_back({k, v, read + 1});
      }
    }
  std::printf("%ld states\n", states);
}
"""


def test_every_copy_in_flight_is_awaited(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) > 1000
