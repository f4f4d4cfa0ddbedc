"""Which rows the norm kernels may read in whole aligned words (no GPU): the library's own function, called by a small
program, against the places of the words themselves."""
from __future__ import annotations

import os
import subprocess

import pytest

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "row_words.cuh"

// Rows, values of a row, stride, in threes: the first row that is not read so, at every place of the matrix in a word.
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const int64_t rows = atoll(argv[i]), cols = atoll(argv[i + 1]), ld = atoll(argv[i + 2]);
    for (uintptr_t at = 0; at < 8; ++at) {
      const auto* p = reinterpret_cast<const uint16_t*>(4096 + 2 * at);
      std::printf("%lld ", (long long)t2s::row::inner_end(t2s::row::view_of(p, ld, rows, cols), rows));
    }
    std::printf("%lld\n", (long long)t2s::row::inner_end(t2s::row::view_of(nullptr, ld, rows, cols), rows));
  }
}
"""
# Around and below a word's eight values; slices of wider tensors; more rows than a block's groups, and fewer.
CASES = [(rows, cols, cols + pad) for rows in (1, 2, 3, 17, 24, 40) for cols in (1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 257, 1003)
         for pad in (0, 1, 2, 5, 8)]


@pytest.fixture(scope="module")
def ends(tmp_path_factory):
    from roofline_driven_tiling_gb300 import build
    folder = tmp_path_factory.mktemp("rows")
    source, program = str(folder / "rows.cu"), str(folder / "rows")
    with open(source, "w") as f:
        f.write(SOURCE)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
                    source, "-o", program], check=True)
    out = subprocess.run([program, *[str(v) for case in CASES for v in case]], check=True, capture_output=True, text=True).stdout
    return [[int(v) for v in line.split()] for line in out.splitlines()]


def test_inner_rows(ends):
    for (rows, cols, ld), (*got, absent) in zip(CASES, ends):
        assert absent == rows
        # A group's later rows: 16 groups share a block where rows are of up to 256 values.
        first = 16 if cols <= 256 else 1
        for at, end in enumerate(got):
            last = at + (rows - 1) * ld + cols  # after the matrix, in values from an aligned place
            for r in range(first, end):
                begin = (at + r * ld) // 8 * 8
                beyond = -(-(at + r * ld + cols) // 8) * 8
                assert at <= begin and beyond <= last, (rows, cols, ld, at, r)
        # Kept out are the last row, or as many as seven values span.
        assert got == [rows - (0 if rows == 1 else 1 if ld >= 7 else -(-7 // ld))] * 8
