"""Grid sizes of the persistent row-wise kernels, for any number of blocks that fit on the device (a part of a GPU has
few): the host rule of csrc/row_grid.h, compiled by the host compiler. No GPU is needed."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_ffn_backward_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "row_grid.h"
int main() {
  for (long fit = 1; fit <= 40; ++fit)
    for (long need = 1; need <= 100; ++need)
      for (long multiple = 1; multiple <= 8; multiple *= 2)
        std::printf("%ld %ld %ld %ld\n", fit, need, multiple, (long)swg::persistent_blocks(fit, need, multiple));
}
"""


@pytest.fixture(scope="module")
def cases(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("grid")
    (d / "grid.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(d / "grid.cpp"), "-o", str(d / "grid")], check=True)
    out = subprocess.run([str(d / "grid")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_a_groups_rows_lie_a_multiple_apart(cases):
    assert len(cases) == 40 * 100 * 4
    for fit, need, multiple, blocks in cases:
        assert 0 <= blocks <= min(fit, need)
        # block b takes rows b, b + blocks, ... of `need`
        if blocks and need > blocks:
            assert blocks % multiple == 0, (fit, need, multiple, blocks)


def test_none_only_where_too_few_fit(cases):
    for fit, need, multiple, blocks in cases:
        assert (blocks == 0) == (need > fit and fit < multiple), (fit, need, multiple, blocks)
        if multiple == 1:
            assert blocks == min(fit, need)
