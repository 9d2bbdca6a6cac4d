"""How qgemm_i8 cuts a product: its rule compiled for the host, over products of every size."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SMS, OF2, OF4 = 148, 74, 33  # of a B200: SMs, and clusters of 2 and 4 whole SMs that run at once
PROGRAM = """
#include <cstdio>
#include "i8_cut.h"
int main() {
  int t, n, k, sms, of2, of4;
  while (scanf("%d %d %d %d %d %d", &t, &n, &k, &sms, &of2, &of4) == 6) {
    const bqg::I8Cut c = bqg::i8_cut(t, n, k, sms, bqg::I8Clusters{of2, of4});
    printf("%d %d\\n", c.tokens, c.split);
  }
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("i8_cut")
    (at / "cut.cpp").write_text(PROGRAM)
    exe = str(at / "cut")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "block_quant_gemv_b200", "csrc"), str(at / "cut.cpp"), "-o", exe], check=True)

    def run(shapes, of2=OF2, of4=OF4):
        text = "".join(f"{t} {n} {k} {SMS} {of2} {of4}\n" for t, n, k in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


SHAPES = [(t, n, k) for t in (1, 3, 9, 16, 17, 40, 64, 100, 128, 129, 300, 1000, 8192) for k in (16, 128, 129, 2051, 4096, 65536)
          for n in list(range(1, 10000, 389)) + [128 * m for m in (1, 32, 33, 34, 36, 37, 38, 64, 74, 75, 148)] + [14336]]


@pytest.mark.parametrize("of2,of4", [(OF2, OF4), (60, 20), (0, 0)])
def test_clusters_that_share_k_all_run_at_once(cut, of2, of4):
    for (t, n, k), (bn, split) in zip(SHAPES, cut(SHAPES, of2, of4)):
        assert bn in (16, 32, 64, 128, 256, 512) and split in (1, 2, 4), (t, n, k)
        tiles = -(-n // 128) * -(-t // bn)
        if split > 1:
            assert bn <= 128 and split <= -(-k // 128), (t, n, k)
            assert tiles <= {2: of2, 4: of4}[split], (t, n, k, bn, split)


def test_known_cuts(cut):
    shapes = [(16, 4224, 4096), (16, 4352, 4096), (16, 4736, 4096), (24, 4096, 4096), (8192, 14336, 4096), (128, 14336, 4096)]
    assert cut(shapes) == [(16, 4), (16, 2), (16, 2), (32, 4), (512, 1), (128, 1)]


def test_the_most_rows(cut):
    most = 2 ** 31 - 512
    for bn, split in cut([(most, 1, 16), (9, most, 16), (most, most, 65536)]):
        assert bn >= 16 and split == 1
