"""How the 8-bit and grouped products are cut up, before any device work: the
rules of csrc/plans.h, compiled for the host and asked for the sizes that the
GPU tests run, so that every way of running them is known to be tested."""
import os
import shutil
import subprocess

import pytest

import tile_size_selection_amd as tss

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tile_size_selection_amd", "csrc")
DRIVER = """
#include <cstdio>
#include <initializer_list>
#include "plans.h"
int main() {
  char what;
  long long a, b, c, e;
  while (std::scanf(" %c %lld %lld %lld %lld", &what, &a, &b, &c, &e) == 5) {
    if (what == 'p' || what == 'g') {
      for (bool exact : {false, true}) {
        const tss::ProductPlan p = what == 'p' ? tss::plan_product(a, b, c, exact) : tss::plan_grouped_fp8(a, b, c, e, exact);
        int n = 1, k;
        if (what == 'p') tss::split_ranges(c, p.splits, &n, &k);
        std::printf("%d %d %d ", p.bm, n, p.sets);
      }
      std::printf("\\n");
    } else {
      std::printf("%d %d\\n", tss::plan_grouped_rows(a, b, e), tss::plan_grad_b(a, e));
    }
  }
}
"""

# M, N, K whose K is cut into ranges; M N is odd in some, and not a multiple of 4 in others
SPLIT = [(1001, 1001, 4112), (515, 521, 8208), (700, 1003, 2064), (513, 510, 8192), (512, 512, 8192)]

# M, N, K of gemm_fp8: (tile rows, ranges of K, sets of waves) for 16-bit outputs, and for fp32 sums
PRODUCTS = {
    (16, 16, 128): ((16, 1, 1), (16, 1, 1)), (100, 1000, 4112): ((16, 1, 1), (16, 1, 1)),
    (1500, 1210, 144): ((64, 1, 1), (64, 1, 1)), (1100, 1003, 528): ((64, 1, 1), (64, 1, 1)),
    (900, 1201, 1040): ((64, 1, 1), (64, 1, 2)), (1300, 1030, 2064): ((64, 1, 2), (64, 1, 2)),
    (1001, 1001, 4112): ((64, 2, 2), (64, 2, 2)), (515, 521, 8208): ((64, 5, 1), (64, 5, 2)),
    (700, 1003, 2064): ((64, 2, 1), (64, 2, 2)), (513, 510, 8192): ((64, 7, 1), (64, 7, 2)),
    (512, 512, 8192): ((64, 8, 1), (64, 8, 2)),
    (1700, 1704, 272): ((128, 1, 1), (64, 1, 1)), (1700, 1701, 1040): ((128, 1, 1), (64, 1, 1)),
    (2101, 2105, 272): ((256, 1, 1), (128, 1, 1)), (4096, 4096, 128): ((256, 1, 1), (128, 1, 1)),
}

# T, the groups' sizes, K, N of gemm_grouped_fp8: (tile rows, 1, sets of waves) as above
GROUPED = {
    (70, (17, 0, 33, 20), 400, 520): ((16, 1, 1), (16, 1, 1)),
    (700, (60, 0, 70, 130, 0, 1, 64, 128, 90, 65, 33, 47), 144, 2056): ((64, 1, 1), (64, 1, 1)),
    (700, (300, -5, 270), 2064, 1032): ((64, 1, 1), (64, 1, 2)),
    (300, (130, 0, 150), 4112, 1032): ((64, 1, 2), (64, 1, 2)),
    (520, (100, 129, 0, 260, 3), 272, 4104): ((128, 1, 1), (128, 1, 1)),
    (1200, (200, 0, 300, 1, 250, 127, 128, 150), 144, 4104): ((128, 1, 1), (128, 1, 1)),
    (1200, (400, 650), 272, 4104): ((256, 1, 1), (128, 1, 1)),
}


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plans")
    (d / "driver.cpp").write_text(DRIVER)
    subprocess.run([cxx, "-std=c++20", "-I", CSRC, "-o", str(d / "driver"), str(d / "driver.cpp")], check=True)

    def f(lines):
        r = subprocess.run([str(d / "driver")], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
    return f


def test_every_way_of_a_product_is_tested(ask):
    got = ask([f"p {M} {N} {K} 0" for M, N, K in PRODUCTS])
    assert [(g[:3], g[3:]) for g in got] == list(PRODUCTS.values())
    for half in (0, 1):  # a new way wants a size here
        assert {(w[half][0], w[half][1] > 1, w[half][2]) for w in PRODUCTS.values()} >= \
            {(16, False, 1), (64, False, 1), (64, False, 2), (64, True, 2), (128, False, 1)}
    assert all(s in PRODUCTS and PRODUCTS[s][0][1] > 1 for s in SPLIT)


def test_every_way_of_a_grouped_8_bit_product_is_tested(ask):
    got = ask([f"g {T} {N} {K} {len(sizes)}" for T, sizes, K, N in GROUPED])
    assert [(g[:3], g[3:]) for g in got] == list(GROUPED.values())


def test_every_way_of_a_grouped_16_bit_product_is_tested(ask):
    from test_ops_gemm_gpu import CASES
    cases = [(T, len(sizes), K, N) for (T, sizes), (K, N) in CASES]
    forward = ask([f"f {T} {N} {K} {E}" for T, E, K, N in cases])
    grad_a = ask([f"f {T} {K} {N} {E}" for T, E, K, N in cases])
    assert {f[0] for f in forward} == {f[0] for f in grad_a} == {16, 64, 256}
    assert {f[1] for f in forward} == {128, 256}


@pytest.mark.parametrize("size", PRODUCTS)
def test_workspace_is_the_ranges_partial_sums(size):
    M, N, K = size
    n = max(way[1] for way in PRODUCTS[size])
    # each range's slice starts on a 16-byte border
    assert tss.gemm_fp8_workspace_size(M, N, K) == (n * ((M * N + 3) // 4 * 16) if n > 1 else 0)
