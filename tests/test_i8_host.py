"""int8 rows and their product on the host: the oracle's pins, and every refusal of the two calls
(C ABI and binding), all before any launch."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import i8 as oi

A = 0x10000  # a fake device address; nothing is dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    from block_quant_gemv_b200 import build
    build.build()
    import block_quant_gemv_b200 as bqg
    return bqg


# ---------------------------------------------------------------- oracle pins
def test_hand_row():
    # max 127 -> scale 1: the values round to themselves, halves go to the even integer
    q, s = oi.quantize_rows(np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0, 3.49]], np.float32))
    assert s[0] == 1.0
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, -127, 3]


def test_zero_tiny_and_nonfinite_rows():
    x = np.zeros((5, 4), np.float32)
    x[1, 2] = 1e-31          # scale 7.9e-34, below 2^-100
    x[2, 0] = np.inf
    x[3, 1] = np.nan
    x[4, 3] = -2.0 ** -90
    q, s = oi.quantize_rows(x)
    assert s[0] == 0 and s[1] == 0 and not q[:4].any()
    assert np.isnan(s[2]) and np.isnan(s[3])
    assert s[4] > 0 and q[4].tolist() == [0, 0, 0, -127]


@pytest.mark.parametrize("seed", range(4))
def test_quantize_agrees_with_rationals(seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((6, 40)).astype(np.float32)
    x = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)  # bf16 values: exact ties occur
    x[0, 0], x[0, 1:20] = 127.0, r.integers(-253, 254, 19) / 2.0      # scale 1: halves
    q, s = oi.quantize_rows(x)
    for t in range(6):
        want = Fraction(float(np.max(np.abs(x[t])))) / 127
        assert abs(Fraction(float(s[t])) - want) <= want * Fraction(1, 2 ** 24)
        assert q[t].tolist() == [oi.round_exact(v, s[t]) for v in x[t]]


def test_product_is_the_naive_sum():
    r = np.random.default_rng(5)
    q, w = r.integers(-128, 128, (3, 7)), r.integers(-128, 128, (4, 7))
    sx, sw, b = r.random(3), r.random(4), r.random(4)
    y = oi.product(q, sx, w, sw, b)
    for t in range(3):
        for n in range(4):
            assert y[t, n] == pytest.approx(sum(int(q[t, i]) * int(w[n, i]) for i in range(7)) * sx[t] * sw[n] + b[n],
                                            rel=1e-14)


# ---------------------------------------------------------------- refusals of the C ABI
def test_quantize_argument_errors(L):
    f = L.lib().quantize_rows_i8
    assert f(2, None, 64, A, 64, A, 1, 64, None) == -1
    assert f(2, A, 64, None, 64, A, 1, 64, None) == -1
    assert f(2, A, 64, A, 64, None, 1, 64, None) == -1
    assert f(2, A, 64, A, 64, A, 0, 64, None) == -1          # no rows
    assert f(2, A, 64, A, 64, A, 1, 0, None) == -1           # no columns
    assert f(0, A, 64, A, 64, A, 1, 64, None) == -1          # unknown type
    assert f(4, A, 64, A, 64, A, 1, 64, None) == -1
    assert f(2, A, 1 << 20, A, 1 << 20, A, 1, L.MAX_I8_COLS + 1, None) == -8
    assert f(2, A, 63, A, 64, A, 1, 64, None) == -3          # ldx below k
    assert f(2, A, 64, A, 48, A, 1, 64, None) == -3          # ldq below k
    assert f(2, A, 64, A, 72, A, 1, 64, None) == -3          # ldq not a multiple of 16
    assert f(2, A + 1, 64, A, 64, A, 1, 64, None) == -4      # X below its element's alignment
    assert f(1, A + 2, 64, A, 64, A, 1, 64, None) == -4
    assert f(2, A, 64, A + 8, 64, A, 1, 64, None) == -4      # Xq not 16-byte aligned
    assert f(2, A, 64, A, 64, A + 2, 1, 64, None) == -4


def test_product_argument_errors(L):
    f = L.lib().qgemm_i8
    ok = [A, 64, A, A, 64, A, None, 2, A, 100, 3, 100, 64, None]

    def call(**change):
        names = ["X", "ldx", "sx", "W", "ldw", "sw", "bias", "out", "Y", "ldy", "tokens", "n", "k", "stream"]
        return f(*[change.get(n, v) for n, v in zip(names, ok)])
    for name in ("X", "sx", "W", "sw", "Y"):
        assert call(**{name: None}) == -1, name
    for name in ("tokens", "n", "k"):
        assert call(**{name: 0}) == -1, name
    assert call(out=0) == -1 and call(out=4) == -1
    assert call(k=L.MAX_I8_COLS + 1, ldx=1 << 20, ldw=1 << 20) == -8
    assert call(ldx=48) == -3 and call(ldw=48) == -3 and call(ldy=99) == -3
    assert call(ldx=72) == -3 and call(ldw=72) == -3          # pitches of whole 16 bytes
    assert call(X=A + 8) == -4 and call(W=A + 8) == -4
    assert call(sx=A + 2) == -4 and call(sw=A + 2) == -4 and call(bias=A + 2) == -4
    assert call(Y=A + 1) == -4 and call(out=1, Y=A + 2) == -4


def test_valid_calls_without_gpu_fail_loudly(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.lib().quantize_rows_i8(2, A, 64, A, 64, A, 1, 64, None) in (-6, -7)
    assert L.lib().qgemm_i8(A, 64, A, A, 64, A, None, 2, A, 100, 3, 100, 64, None) in (-6, -7)


def test_limit_matches_header(L):
    import os
    import re
    from tests.conftest import ROOT
    m = re.search(r"#define BQG_MAX_I8_COLS (\d+)", open(os.path.join(ROOT, "include", "bqg.h")).read())
    assert int(m.group(1)) == L.MAX_I8_COLS
    # any int8 values: 128 * 128 * k stays inside int32
    assert 128 * 128 * L.MAX_I8_COLS < 2 ** 31


# ---------------------------------------------------------------- refusals of the binding
def test_binding_refuses_host_tensors(L):
    with pytest.raises(TypeError):
        L.quantize_rows_i8(torch.zeros(2, 32))
    q = torch.zeros(2, 32, dtype=torch.int8)
    with pytest.raises(TypeError):
        L.qgemm_i8(q, torch.ones(2), q, torch.ones(2))
