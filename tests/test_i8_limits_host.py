"""The most rows of the int8 calls, refused before any launch: past it the index of a tile's last row would
not fit 32 bits, and a call would leave its outputs as they were."""
import os
import re

import pytest

from tests.conftest import ROOT

A = 0x10000  # a fake device address; nothing is dereferenced on these paths
LARGEST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    from block_quant_gemv_b200 import build
    build.build()
    import block_quant_gemv_b200 as bqg
    return bqg


def test_limit_matches_header(L):
    m = re.search(r"#define BQG_MAX_I8_ROWS (\d+)", open(os.path.join(ROOT, "include", "bqg.h")).read())
    assert int(m.group(1)) == L.MAX_I8_ROWS
    assert L.MAX_I8_ROWS + 256 + 255 <= LARGEST  # a tile that starts at the last row, plus its rounding up


@pytest.mark.parametrize("over", [1, 257, 511])
def test_more_rows_are_refused(L, over):
    rows = L.MAX_I8_ROWS + over
    lib = L.lib()
    assert lib.quantize_rows_i8(2, A, 64, A, 64, A, rows, 64, None) == -8
    assert lib.qgemm_i8(A, 64, A, A, 64, A, None, 2, A, 100, rows, 100, 64, None) == -8
    assert lib.qgemm_i8(A, 64, A, A, 64, A, None, 2, A, rows, 3, rows, 64, None) == -8
