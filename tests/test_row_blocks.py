"""The copy of 16-bit rows whose starts are off 16-byte boundaries reads the
aligned blocks that the rows lie in.  On the host, for every alignment and for
rows from one element on: each block that the copy reads, as it chooses them
by row_blocks.h, lies inside the matrix."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

import dense_gemm_tensor_tcgen05_gb300 as g

PROGRAM = r"""
#include <cstdio>
#include "row_blocks.h"
using namespace gb300;

static long outside = 0, whole = 0;

static void read(uintptr_t a, uintptr_t bytes, uintptr_t lo, uintptr_t hi) {
    if (a < lo || a + bytes > hi) ++outside;
}

int main() {
    for (uintptr_t base = 4096; base < 4112; base += 2)
        for (int64_t cols = 1; cols <= 40; ++cols)
            for (int64_t ld = cols; ld <= cols + 9; ++ld)
                for (int64_t rows = 1; rows <= 24; ++rows) {
                    const uintptr_t lo = base, hi = base + 2 * ((rows - 1) * ld + cols);
                    for (int64_t i = 0; i < rows; ++i) {
                        const uintptr_t from = base + 2 * i * ld;
                        const bool direct = row_inside(from, cols, lo, hi);
                        whole += direct;
                        for (int64_t c = 0; c < cols; c += 8) {
                            const uintptr_t at = from + 2 * c, block = at - (at & 15);
                            const int64_t valid = cols - c;
                            if (direct) {                              // the row's blocks, two to a chunk
                                read((from - (from & 15)) + 2 * c, 32, lo, hi);
                            } else if (valid >= 8 && (at & 15) == 0) {
                                read(at, 16, lo, hi);
                            } else if (pair_inside(at, lo, hi)) {
                                read(block, 32, lo, hi);
                            } else {                                   // one by one
                                read(at, 2 * (valid < 8 ? valid : 8), lo, hi);
                            }
                        }
                    }
                }
    std::printf("%ld %ld\n", outside, whole);
    return 0;
}
"""


def test_blocks_read_lie_inside_the_matrix(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    csrc = os.path.join(os.path.dirname(g.__file__), "csrc")
    src, exe = tmp_path / "blocks.cpp", tmp_path / "blocks"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", f"-I{csrc}", str(src), "-o", str(exe)], check=True)
    outside, whole = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert outside == 0
    assert whole > 0            # rows well inside are still read block by block
