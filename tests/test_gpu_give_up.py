"""A bounded wait of moe_layer that runs out: the call ends, reports BQG_DEVERR_TIMEOUT, leaves its state
words zero, and the next call on the same workspace is right.  A barrier's counter starts one below zero
(every CTA counts on it before it waits), so that it never reaches the grid's size."""
import time

import pytest
import torch

import block_quant_gemv_b200 as bqg
from synth import workloads as wl
from tests.moe_util import device_layer
from tests.test_gpu_moe_layer import SMALL, check, router
from tests.util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spec,tokens,barrier", [(SMALL[0], 1, 1), (SMALL[0], 4, 0), (SMALL[0], 4, 1),
                                                 (wl.GEMMA_MOE, 1, 1), (wl.GEMMA_MOE, 4, 1), (wl.GEMMA_MOE, 8, 2)],
                         ids=lambda v: v.name if hasattr(v, "name") else str(v))
def test_a_barrier_that_never_completes(spec, tokens, barrier):
    need_gpu()
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    x, R = wl.moe_tokens(spec, 0, tokens), router(spec, 0)
    ws = bqg.moe_layer_workspace(L, tokens)
    state = ws[:bqg.MOE_LAYER_STATE_BYTES].view(torch.int32)
    x_dev, R_dev = x.cuda(), R.cuda()
    bqg.moe_layer(L, R_dev, x_dev, workspace=ws)
    assert bqg.bqg_device_errors() == 0
    state[32 * barrier] = -1
    torch.cuda.synchronize()
    t0 = time.time()
    bqg.moe_layer(L, R_dev, x_dev, workspace=ws)
    bits = bqg.bqg_device_errors()  # synchronises, reads and clears
    assert bits == bqg.DEVERR_TIMEOUT
    assert 1.5 < time.time() - t0 < 60
    assert not state.any()
    y, idx, w = bqg.moe_layer(L, R_dev, x_dev, workspace=ws)
    assert bqg.bqg_device_errors() == 0
    check(spec, x, R, y, idx, w)
