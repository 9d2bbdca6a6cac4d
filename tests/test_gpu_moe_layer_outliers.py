"""GPU parity of moe_layer on rows with one value far above the others whose weights are zero, so that it adds
nothing to y, and on rows of very small values.

Bound: x and h are fixed point per row, off by up to 2^-32 of the row's largest value.  At a value R times
the others' root mean square each of a sum's terms is off by 2^-32 R / sqrt(3) of that (root mean square,
either sign): 1.3e-6 at R = 1e4, and sqrt(2) times that for gate and up together, in each element of y.
With an fp32 sum's own error (3.6e-6 of max|y|, as for rows without outliers) that is below 1e-5 of max|y|."""
import numpy as np
import pytest
import torch

import block_quant_gemv_b200 as bqg
from oracle import moe as om
from synth import workloads as wl
from tests.moe_util import device_layer
from tests.test_gpu_moe_layer import router
from tests.util import assert_close, need_gpu

pytestmark = pytest.mark.gpu
TOL = 1e-5
Q8, Q4, I4, I2 = bqg.Q8_0, bqg.Q4_0, bqg.I4_ROW, bqg.I2_ROW
PER_BYTE = {Q8: 1, Q4: 2, I4: 2, I2: 4}
BLOCK = {Q8: 34, Q4: 18}


def zero_column(buf, fmt, rows, cols, c):
    """The weights of column c become zero (buf: one matrix's bytes)."""
    if fmt in BLOCK:
        b = buf[:rows * cols // 32 * BLOCK[fmt]].reshape(rows, cols // 32, BLOCK[fmt])
        code, at = b[:, c // 32, 2 + c % 32 // PER_BYTE[fmt]], c % 2
        if fmt == Q8:
            code[:] = 0
            return
        zero = 8
    else:
        code = buf[:rows * cols // PER_BYTE[fmt]].reshape(rows, -1)[:, c // PER_BYTE[fmt]]
        at, zero = c % PER_BYTE[fmt], 0
    bits = 8 // PER_BYTE[fmt]
    code[:] = (code & (255 - (((1 << bits) - 1) << (bits * at)))) | (zero << (bits * at))


def scale_rows(buf, fmt, rows, cols, which, factor):
    """The scales of the rows `which` (a slice or a list) times `factor`."""
    if fmt in BLOCK:
        d = buf[:rows * cols // 32 * BLOCK[fmt]].reshape(rows, cols // 32, BLOCK[fmt])
        raw = np.ascontiguousarray(d[which, :, :2])
        d[which, :, :2] = (raw.view(np.float16) * np.float16(factor)).view(np.uint8)
    else:
        at = (rows * cols // PER_BYTE[fmt] + 15) // 16 * 16
        s = buf[at:at + 4 * rows].view(np.float32)
        s[which] *= np.float32(factor)


class Edited:
    """A layer on the host whose matrices a test may change, then the device layer and the oracle's."""

    def __init__(self, spec):
        self.spec, self.T = spec, wl.build_moe_layer(spec, 0, 0, device="cpu")

    def matrices(self, name):
        """(bytes, fmt, rows, cols) of every matrix called `name`, the shared expert's too."""
        s = self.spec
        stride, buf = getattr(self.T, name + "_stride"), getattr(self.T, name).numpy()
        for e in range(s.n_experts):
            r, c = (s.hidden, s.inter) if name == "down" else (s.inter, s.hidden)
            yield buf[e * stride:(e + 1) * stride], s.expert_fmt, r, c
        if self.T.shared is not None:
            r, c = (s.hidden, s.shared_inter) if name == "down" else (s.shared_inter, s.hidden)
            yield self.T.shared[("gate", "up", "down").index(name)].numpy(), s.shared_fmt, r, c

    def device(self):
        T = self.T
        return device_layer(wl.MoETensors(T.spec, T.gate.cuda(), T.up.cuda(), T.down.cuda(), T.gate_stride, T.up_stride,
                                          T.down_stride, None if T.shared is None else tuple(t.cuda() for t in T.shared)))

    def oracle(self):
        s, mats = self.spec, {n: [m for m, *_ in self.matrices(n)] for n in ("gate", "up", "down")}
        size = {n: bqg.bqg_weight_bytes(s.expert_fmt, *((s.hidden, s.inter) if n == "down" else (s.inter, s.hidden)))
                for n in mats}

        def expert(e):
            return om.Expert(s.expert_fmt, *[mats[n][e][:size[n]] for n in ("gate", "up", "down")])
        shared = om.Expert(s.shared_fmt, *[mats[n][-1] for n in ("gate", "up", "down")]) if s.shared_inter else None
        return om.Layer(s.n_experts, s.top_k, s.hidden, s.inter, s.act, expert, shared, s.shared_inter)


def check(layer, x, R):
    need_gpu()
    L, OL = layer.device(), layer.oracle()
    for tokens in (1, x.shape[0]):
        xt = x[:tokens]
        y, idx, w = bqg.moe_layer(L, R.cuda(), xt.cuda())
        assert bqg.bqg_device_errors() == 0
        ridx, rw = om.router_topk(om.router_logits(R.numpy(), xt.numpy()), layer.spec.top_k)
        assert np.array_equal(idx.cpu().numpy(), ridx)
        assert_close(w, rw, tol=1e-5)
        assert_close(y, om.moe_layer(OL, xt.numpy(), ridx, rw), tol=TOL)


SPECS = [
    wl.MoESpec("o_q4_shared_q8", 8, 2, 512, 256, Q4, bqg.ACT_GELU_TANH, 192, Q8),
    wl.MoESpec("o_q8", 6, 3, 480, 320, Q8, bqg.ACT_SILU),
    wl.MoESpec("o_i4_shared_q4", 16, 8, 768, 256, I4, bqg.ACT_SILU, 128, Q4),
    wl.MoESpec("o_i2_shared_i4", 9, 4, 640, 320, I2, bqg.ACT_GELU_TANH, 128, I4),
]


@pytest.mark.parametrize("spec", SPECS, ids=lambda s: s.name)
@pytest.mark.parametrize("outlier", [1e3, 1e4])
def test_outlier_of_x_under_zero_weights(spec, outlier):
    layer, x, R = Edited(spec), wl.moe_tokens(spec, 1, 4), router(spec, 0)
    for t, c in enumerate((0, 37, spec.hidden // 2, spec.hidden - 1)):
        x[t, c] = outlier if t % 2 else -outlier
        R[:, c] = 0
        for name in ("gate", "up"):
            for m in layer.matrices(name):
                zero_column(*m, c)
    check(layer, x, R)


@pytest.mark.parametrize("spec", SPECS, ids=lambda s: s.name)
def test_outlier_of_h_under_zero_weights(spec):
    layer, x, R = Edited(spec), wl.moe_tokens(spec, 2, 4), router(spec, 0)
    for f in (3, 32, 77, 127):
        for name in ("gate", "up"):
            for m in layer.matrices(name):
                scale_rows(*m, [f], 30)
        for m in layer.matrices("down"):
            zero_column(*m, f)
    check(layer, x, R)


@pytest.mark.parametrize("power", [-100, -115])
def test_rows_of_very_small_values(power):
    """x far below 2^-96 (where the fixed point's factor alone is beyond fp32) with weights that make up for it."""
    spec = SPECS[3]
    plain = wl.MoESpec("o_i2", spec.n_experts, spec.top_k, spec.hidden, spec.inter, I2, spec.act)
    layer, x, R = Edited(plain), wl.moe_tokens(plain, 3, 4), router(plain, 0)
    x *= 2.0 ** power
    R *= 2.0 ** -power
    for name in ("gate", "up"):
        for m in layer.matrices(name):
            scale_rows(*m, slice(None), 2.0 ** -power)
    check(layer, x, R)
