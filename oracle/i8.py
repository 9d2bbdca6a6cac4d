"""Oracle of int8 row quantization and of the scaled int8 product, in exact arithmetic where it can
be: the scale is the fp32 nearest to max|row| / 127, the quotient is compared in rationals, the
sums are int64, the scaling is float64.  Test infrastructure only."""
import math
from fractions import Fraction

import numpy as np

TINY = 2.0 ** -100


def scale_of(row) -> np.float32:
    """The scale of one row (any float type): NaN when it holds an Inf or a NaN, 0 below 2^-100."""
    row = np.asarray(row, np.float64)
    if not np.all(np.isfinite(row)):
        return np.float32(np.nan)
    # float64 of an fp32 (or narrower) value over 127, rounded to fp32: the double rounding is
    # harmless, since a quotient by 127 is never within 2^-53 of a 25-bit midpoint unless exact
    s = np.float32(np.max(np.abs(row)) / 127.0)
    return s if s >= TINY else np.float32(0)


def quantize_rows(x):
    """(q int8, scale fp32) of rows x, vectorised in float64.  x / s in float64 is exact to 2^-53,
    and a true tie (2 x = (2m + 1) s) is found exactly, since both products are."""
    x = np.asarray(x, np.float64)
    s = np.array([scale_of(r) for r in x], np.float32)
    q = np.zeros(x.shape, np.int8)
    for t in range(x.shape[0]):
        if not s[t] > 0:
            continue
        st = np.float64(s[t])
        f = np.floor(x[t] / st)
        f = np.where((f + 1) * st <= x[t], f + 1, f)
        f = np.where(f * st > x[t], f - 1, f)
        up = 2 * x[t] - (2 * f + 1) * st      # exact in float64: 24-bit numbers times 9-bit integers
        r = np.where((up > 0) | ((up == 0) & (f % 2 != 0)), f + 1, f)
        q[t] = r.astype(np.int8)
    return q, s


def round_exact(x: float, s: float) -> int:
    """x / s to the nearest integer, ties to even, in rationals."""
    v = Fraction(float(x)) / Fraction(float(s))
    f = math.floor(v)
    d = v - f
    if d > Fraction(1, 2) or (d == Fraction(1, 2) and f % 2):
        return f + 1
    return f


def sums(q, w):
    """Exact integer sums [tokens, n]."""
    return np.asarray(q, np.int64) @ np.asarray(w, np.int64).T


def product(q, sx, w, sw, bias=None):
    y = sums(q, w).astype(np.float64) * np.asarray(sx, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
    return y if bias is None else y + np.asarray(bias, np.float64)[None, :]
