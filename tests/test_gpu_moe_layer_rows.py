"""GPU parity of moe_layer on rows whose values differ widely: x and h are fixed point per row, so that a
value is off by up to 2^-23 of its row's largest.  A sum over K = 256 such errors, of either sign, is
about sqrt(256) 2^-24 of the largest product, 1e-6 of y, which the largest values dominate as well; the
bound is the call's 1e-5 of max|y|."""
import pytest
import torch

import block_quant_gemv_b200 as bqg
from synth import workloads as wl
from tests.moe_util import device_layer
from tests.test_gpu_moe_layer import SMALL, check, router
from tests.util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spec", [SMALL[i] for i in (0, 2, 4, 5, 6, 7)], ids=lambda s: s.name)
@pytest.mark.parametrize("kind", ["outlier", "tiny", "huge"])
def test_rows_of_any_range(spec, kind):
    need_gpu()
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    x, R = wl.moe_tokens(spec, 3, 4), router(spec, 0)
    if kind == "outlier":
        x[torch.arange(4), torch.tensor([0, 5, spec.hidden // 2, spec.hidden - 1])] = torch.tensor([40., -300., 1000., -77.])
    else:
        x *= 1e-12 if kind == "tiny" else 1e6
        R /= 1e-12 if kind == "tiny" else 1e6   # logits as far apart as before
    for tokens in (1, 4):
        y, idx, w = bqg.moe_layer(L, R.cuda(), x[:tokens].cuda())
        assert bqg.bqg_device_errors() == 0
        check(spec, x[:tokens], R, y, idx, w)


def test_every_token_picks_the_same_expert():
    """Eight equal tokens: an expert's items hold all of them, four passes of two."""
    need_gpu()
    for spec in (SMALL[1], SMALL[3], SMALL[5], SMALL[7]):
        L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
        x, R = wl.moe_tokens(spec, 1, 1).repeat(8, 1).contiguous(), router(spec, 0)
        y, idx, w = bqg.moe_layer(L, R.cuda(), x.cuda())
        assert (idx == idx[0]).all() and (w == w[0]).all() and (y == y[0]).all()
        check(spec, x, R, y, idx, w)
        y1, idx1, w1 = bqg.moe_layer(L, R.cuda(), x[:1].cuda())
        assert torch.equal(idx1, idx[:1])
        assert (y1 - y[:1]).abs().max() <= 1e-5 * y1.abs().max()
