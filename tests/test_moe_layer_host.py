"""Refusals of moe_layer and the size of its workspace, before any launch."""
import ctypes

import pytest

from synth import workloads as wl
from tests.test_abi import _layer_c

A = 0x10000


@pytest.fixture(scope="module")
def L():
    from block_quant_gemv_b200 import build
    build.build()
    import block_quant_gemv_b200 as bqg
    return bqg


def test_limits_match_header(L):
    import os
    import re
    from tests.conftest import ROOT
    text = open(os.path.join(ROOT, "include", "bqg.h")).read()
    for name, val in (("BQG_MOE_LAYER_MAX_TOKENS", L.MOE_LAYER_MAX_TOKENS),
                      ("BQG_MOE_LAYER_STATE_BYTES", L.MOE_LAYER_STATE_BYTES)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == val


def test_workspace_size(L):
    size = L.lib().moe_layer_workspace_size
    for spec in (wl.GEMMA_MOE, wl.GLM_MOE):
        c = _layer_c(spec)
        got = [size(ctypes.byref(c), t) for t in range(1, L.MOE_LAYER_MAX_TOKENS + 1)]
        assert got[0] >= L.MOE_LAYER_STATE_BYTES and all(a <= b for a, b in zip(got, got[1:]))
        assert size(ctypes.byref(c), 0) == 0 and size(ctypes.byref(c), L.MOE_LAYER_MAX_TOKENS + 1) == 0
    c.hidden = 2820
    assert size(ctypes.byref(c), 1) == 0
    assert size(None, 1) == 0


def test_argument_errors(L):
    f = L.lib().moe_layer
    c = _layer_c(wl.GEMMA_MOE)
    at = ctypes.addressof(c)
    need = L.lib().moe_layer_workspace_size(ctypes.byref(c), 2)

    def call(layer=at, R=A, x=A, y=A, idx=A, w=A, tokens=2, ws=A, size=need):
        return f(layer, R, x, y, idx, w, tokens, ws, size, None)
    assert call(layer=None) == -1
    for name in ("R", "x", "y"):
        assert call(**{name: None}) == -1, name
    assert call(idx=None) == -1 and call(w=None) == -1       # one of the two routing outputs
    assert call(tokens=0) == -1
    assert call(tokens=9) == -8
    assert call(R=A + 4) == -4 and call(x=A + 4) == -4 and call(y=A + 2) == -4
    assert call(idx=A + 2) == -4 and call(w=A + 2) == -4
    assert call(size=need - 1) == -5 and call(ws=None) == -5
    assert call(ws=A + 16) == -4
    c.top_k = 9
    assert call() == -8
    c.top_k, c.expert_fmt = 8, 9
    assert call() == -2
    c.expert_fmt, c.act = 2, 5
    assert call() == -1
    c.act, c.hidden = 1, 2820
    assert call() == -3
    c.hidden = 7200
    assert call() == -8


def test_valid_call_without_gpu_fails_loudly(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    c = _layer_c(wl.GLM_MOE)
    need = L.lib().moe_layer_workspace_size(ctypes.byref(c), 8)
    assert L.lib().moe_layer(ctypes.addressof(c), A, A, A, A, A, 8, A, need, None) in (-6, -7)
