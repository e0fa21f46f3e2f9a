"""How the products of 8-bit integers are cut up, before any device work: the
rule of csrc/plans.h, compiled for the host and asked for the sizes that the GPU
tests run, so that every way of running them is known to be tested."""
import os
import shutil
import subprocess

import pytest

import tile_size_selection_amd as tss

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tile_size_selection_amd", "csrc")
DRIVER = """
#include <cstdio>
#include "plans.h"
int main() {
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const tss::ProductPlan p = tss::plan_int8(m, n, k);
    int r, per;
    tss::split_ranges(k, p.splits, &r, &per);
    const long long tiles = (m + p.bm - 1) / p.bm * ((n + p.bn - 1) / p.bn), rest = tiles % tss::kCUs;
    std::printf("%d %d %d\\n", p.bm, r, p.bm == 256 && rest ? tss::tile_pieces(int(rest), false) : 0);
  }
}
"""

# M, N, K: (tile rows, ranges of K, pieces that a tile of the last round is cut into)
WAYS = {
    (1, 8192, 8192): (16, 1, 0), (16, 256, 512): (16, 1, 0), (100, 1000, 4112): (16, 1, 0),
    (1500, 1210, 144): (64, 1, 0), (1300, 1030, 2064): (64, 1, 0),
    (512, 512, 8192): (64, 5, 0), (515, 521, 8208): (64, 5, 0), (256, 512, 8192): (64, 6, 0), (128, 4096, 4096): (64, 3, 0),
    (700, 1003, 4112): (64, 2, 0), (40, 2000, 131056): (64, 8, 0),
    (1700, 1704, 272): (128, 1, 0), (1700, 1701, 1040): (128, 1, 0),
    (4096, 4096, 128): (256, 1, 0), (2101, 2105, 272): (256, 1, 2), (2300, 1900, 144): (256, 1, 2), (4300, 4100, 144): (256, 1, 4),
    (4200, 4357, 272): (256, 1, 4), (4500, 4600, 160): (256, 1, 2), (4801, 4099, 144): (256, 1, 2), (5000, 5001, 144): (256, 1, 1),
    (2600, 2600, 272): (256, 1, 2), (3000, 5000, 2048): (256, 1, 1),
}


@pytest.fixture(scope="module")
def ways(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plans")
    (d / "driver.cpp").write_text(DRIVER)
    subprocess.run([cxx, "-std=c++20", "-I", CSRC, "-o", str(d / "driver"), str(d / "driver.cpp")], check=True)
    lines = "".join(f"{m} {n} {k}\n" for m, n, k in WAYS)
    r = subprocess.run([str(d / "driver")], input=lines, capture_output=True, text=True, check=True)
    return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]


def test_every_way_of_a_product_is_tested(ways):
    assert ways == list(WAYS.values())
    assert {(w[0], w[1] > 1, w[2]) for w in ways} >= {(16, False, 0), (64, False, 0), (64, True, 0), (128, False, 0),
                                                      (256, False, 0), (256, False, 1), (256, False, 2), (256, False, 4)}


@pytest.mark.parametrize("size", WAYS)
def test_workspace_is_the_ranges_partial_sums(size):
    (M, N, K), n = size, WAYS[size][1]
    # each range's slice starts on a 16-byte border
    assert tss.gemm_int8_workspace_size(M, N, K) == (n * ((M * N + 3) // 4 * 16) if n > 1 else 0)
