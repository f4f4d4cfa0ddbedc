"""The host's planning of the feed-forward products (no GPU): the library's own functions, called by a small
program, on weights' gradients over many rows, which may be cut into many numbers of pieces."""
from __future__ import annotations

import os
import subprocess

import pytest

SOURCE = r"""
#include <algorithm>
#include <chrono>
#include <cstdio>

#include "ff_internal.h"

using namespace t2s::ff;

int main() {
  const int64_t sizes[][3] = {{4096, 4096, 4096}, {65536, 256, 256}, {65536, 64, 64}, {16384, 256, 256}, {1 << 20, 64, 64}};
  for (const auto& s : sizes)
    for (int weights = 1; weights <= 2; ++weights) {
      // The gradients of a linear layer, or of a gated pair.
      Task t[3];
      t[0].M = s[0], t[0].N = s[2], t[0].K = s[1];
      t[0].form = weights == 2 ? kJoined : kLinear;
      for (int i = 1; i <= weights; ++i) t[i].M = s[2], t[i].N = s[1], t[i].K = s[0], t[i].split = true;
      const size_t room = weight_partial_bytes(s[0], s[1], s[2], weights);
      PairPlan plan;
      double best = 1e9;
      for (int batch = 0; batch < 20; ++batch) {
        const auto start = std::chrono::steady_clock::now();
        for (int i = 0; i < 50; ++i) plan = plan_pair(t, 1 + weights, 76, room);
        best = std::min(best, std::chrono::duration<double>(std::chrono::steady_clock::now() - start).count() / 50);
      }
      const PairPlan whole = plan_pair(t, 1 + weights, 76, 0);
      std::printf("%lld %lld %lld %d %.9f %d %d %.6f %.6f %zu\n", (long long)s[0], (long long)s[1], (long long)s[2], weights,
                  best * 1e6, plan.width, plan.splits, plan.cost, whole.cost, room);
    }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    import __graft_entry__
    from roofline_driven_tiling_gb300 import build
    __graft_entry__.build()
    folder = tmp_path_factory.mktemp("plan")
    source, program = str(folder / "plan.cpp"), str(folder / "plan")
    with open(source, "w") as f:
        f.write(SOURCE)
    subprocess.run([build.nvcc(), "-std=c++17", "-O2", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), source,
                    build.LIB, "-Xlinker", "-rpath," + os.path.dirname(build.LIB), "-o", program], check=True)
    out = subprocess.run([program], check=True, capture_output=True, text=True).stdout
    return [[float(v) for v in line.split()] for line in out.splitlines()]


def test_pieces(plans):
    """They are taken where they are expected to be quicker, and their sums fit the workspace's part."""
    for m, n, k, weights, _, width, splits, cost, whole, room in plans:
        tiles = weights * -(-k // 256) * -(-n // width)
        assert cost <= whole
        assert (splits > 1) == (m > 4096)
        if splits > 1:
            assert tiles * splits * 256 * width * 4 <= room and m / splits >= 8 * 64


def test_planning_is_short(plans):
    """With a hundred numbers of pieces to choose from, planning takes no more than 30 times what it takes with
    one (0.1 to 0.2 us): a call of tens of microseconds on the device must not wait for its plan."""
    one = {p[3]: p[4] for p in plans if p[0] == 4096}
    for m, n, k, weights, us, *_ in plans:
        assert us <= 30 * one[weights], "%dx%dx%d: %.2f us, %.2f with one" % (m, n, k, us, one[weights])
