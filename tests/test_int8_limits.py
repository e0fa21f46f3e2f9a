"""The largest products of few rows by 8-bit integers: whatever keeps A and B
below 2 GiB fits a launch, whose threads are 32 bits."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tile_size_selection_amd", "csrc")
DRIVER = """
#include <cstdio>
#include "plans.h"
int main() {
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const tss::Int8RowsLaunch f = tss::int8_rows_launch(m, n, k);
    std::printf("%d %d %lld %d\\n", tss::plan_int8(m, n, k).bn, f.groups, (long long)f.workgroups, f.waves);
  }
}
"""

# N that ends inside 4 columns, inside a group of 16, behind a first group; K of one wave, and of one that waits to join
TWO_GROUPS = [(1, 8191, 8192), (16, 6161, 112), (5, 8209, 128), (7, 8193, 16), (16, 6145, 144), (3, 6159, 272), (2, 16388, 48),
              (40, 2049, 112), (16, 8192, 16)]


def run(tmp_path, sizes):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no C++ compiler")
    (tmp_path / "driver.cpp").write_text(DRIVER)
    subprocess.run([cxx, "-std=c++20", "-I", CSRC, "-o", str(tmp_path / "driver"), str(tmp_path / "driver.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "driver")], input="".join("%d %d %d\n" % s for s in sizes), capture_output=True, text=True, check=True)
    return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]


def test_every_product_of_few_rows_fits_a_launch(tmp_path):
    sizes = [(m, (2 ** 31 - 1) // k, k) for m in (1, 2, 15, 16) for k in (16, 32, 112, 128, 144, 256, 1024, 2048, 2064, 65536, 131056)]
    for (m, n, k), (bn, groups, workgroups, waves) in zip(sizes, run(tmp_path, sizes)):
        assert bn == 16 and waves <= 16 and workgroups * 16 * groups >= n > (workgroups - 1) * 16 * groups
        assert workgroups * waves * 64 < 2 ** 32


def test_the_waves_of_a_launch(tmp_path):
    """One for each 128 of K with two groups of columns (two at least, each joins a group), for each 512 with one; 16 at most."""
    want = {(1, 70000000, 16): (16, 2, 2187500, 2), (16, 8192, 8192): (16, 2, 256, 16), (16, 6161, 112): (16, 2, 193, 2),
            (5, 8209, 128): (16, 2, 257, 2), (5, 8209, 400): (16, 2, 257, 4), (16, 4096, 4096): (16, 1, 256, 8), (1, 1, 16): (16, 1, 1, 1)}
    assert run(tmp_path, want) == list(want.values())


def test_two_groups_of_columns_are_tested(tmp_path):
    assert all(way[:2] == (16, 2) for way in run(tmp_path, TWO_GROUPS))


def test_two_groups_where_one_would_take_a_second_round_of_cus(tmp_path):
    want = {(16, 4096, 4096): 1, (16, 4097, 4096): 2, (1, 5120, 4096): 2, (16, 6143, 512): 2, (32, 2048, 4096): 1, (32, 2049, 4096): 2,
            (64, 1024, 4096): 1, (64, 1025, 4096): 2}
    assert [way[:2] for way in run(tmp_path, want)] == [(16, n) for n in want.values()]
