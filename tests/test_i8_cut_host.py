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
    if (of2 < 0) {
      printf("%d 0\\n", int(bqg::i8_few(t, n, k, sms)));
      continue;
    }
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


@pytest.mark.parametrize("few,shapes", [
    (True, [(1, 512, 512), (1, 14336, 2048), (1, 14336, 4096), (2, 1024, 1024), (2, 1024, 2048), (1, 300, 500),
            (4, 512, 512), (4, 1536, 1536), (3, 256, 2048)]),
    (False, [(1, 4096, 4096), (2, 1024, 8192), (1, 2048, 1023), (1, 256, 8191), (1, 14336, 4090), (4, 300, 500),
             (4, 256, 2048), (4, 14336, 1024), (3, 14336, 4096), (8, 640, 640), (8, 14336, 4096), (8, 256, 2048), (16, 64, 64)])])
def test_who_takes_a_few_tokens(cut, few, shapes):
    """Both sides of the rule as they were measured: at 5 to 8 tokens, long rows or odd ones dp4a loses, by up
    to 2.5 times."""
    assert [f for f, _ in cut(shapes, of2=-1)] == [int(few)] * len(shapes)
