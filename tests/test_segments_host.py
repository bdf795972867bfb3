"""An expert's segment clipped to the rows there are (csrc/segments.cuh): the kernels' own
arithmetic, compiled for the host, over starts and ends of any 32-bit value."""

import itertools
import os
import subprocess

from conftest import ROOT, load_build_module

PROGRAM = r"""
#include <cstdio>
#include "segments.cuh"
int main() {
  int start, end, cap;
  while (std::scanf("%d %d %d", &start, &end, &cap) == 3) {
    int first, rows;
    ep::clip_rows(start, end, cap, first, rows);
    std::printf("%d %d\n", first, rows);
  }
}
"""


def test_segments_of_any_ends(tmp_path):
    lo, hi = -(2**31), 2**31 - 1
    values = [lo, lo + 1, -(2**30), -6, -1, 0, 1, 5, 6, 7, 2**30, hi - 1, hi]
    cases = [(s, e, c) for s, e in itertools.product(values, values) for c in (0, 1, 6, hi)]
    src, exe = tmp_path / "clip.cu", tmp_path / "clip"
    src.write_text(PROGRAM)
    subprocess.run([load_build_module().nvcc(), "-O2", "-std=c++17", "-I",
                    os.path.join(ROOT, "combine_get_layout_gb300", "csrc"), "-o", str(exe),
                    str(src)], check=True)
    text = "".join("%d %d %d\n" % c for c in cases)
    got = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    assert len(cases) == len(got.splitlines())
    for (s, e, cap), line in zip(cases, got.splitlines()):
        first, rows = map(int, line.split())
        lo_row, hi_row = max(s, 0), min(e, cap)
        assert rows == max(0, hi_row - lo_row), (s, e, cap, first, rows)
        assert 0 <= first <= cap and first + rows <= cap
        if rows:
            assert first == lo_row
