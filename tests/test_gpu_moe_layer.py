"""GPU parity of moe_layer (router, selection, experts, shared expert and combine in one kernel)
against the float64 oracle.

Bounds, from the arithmetic of the call: logits and weights are fp32 (1e-5, as for the separate
router).  In y every product sum rounds about 20 times (24-bit x or h, the warp's butterfly, up to 7
slices of a row, scale, weight and combine), each 2^-24 of a partial sum, and h passes through three
such sums: 60 * 2^-24 = 3.6e-6 of the typical magnitude, itself below max|y|.  TOL = 1e-5 of max|y|
leaves room for act(g), which multiplies a relative error of g by at most about 2."""
import ctypes

import numpy as np
import pytest
import torch

import block_quant_gemv_b200 as bqg
from oracle import moe as om
from synth import workloads as wl
from tests.moe_util import device_layer, oracle_layer
from tests.util import assert_close, need_gpu

pytestmark = pytest.mark.gpu
TOL = 1e-5

Q8, Q4, I4, I2 = bqg.Q8_0, bqg.Q4_0, bqg.I4_ROW, bqg.I2_ROW
GELU, SILU = bqg.ACT_GELU_TANH, bqg.ACT_SILU
SMALL = [
    wl.MoESpec("l_q4_shared_q8", 8, 2, 128, 64, Q4, GELU, 96, Q8),
    wl.MoESpec("l_q8", 6, 3, 96, 160, Q8, SILU),
    wl.MoESpec("l_i4", 16, 8, 256, 64, I4, SILU),
    wl.MoESpec("l_q4_odd", 5, 5, 160, 96, Q4, GELU, 32, Q4),
    wl.MoESpec("l_i4_shared_q8", 12, 4, 192, 128, I4, GELU, 64, Q8),
    wl.MoESpec("l_i2", 16, 8, 256, 128, I2, SILU),
    wl.MoESpec("l_q4_shared_i2", 8, 2, 128, 64, Q4, GELU, 192, I2),
    wl.MoESpec("l_i2_shared_i4", 9, 1, 320, 192, I2, GELU, 128, I4),
    wl.MoESpec("l_q8_shared_q4", 33, 7, 1056, 352, Q8, SILU, 544, Q4),
    wl.MoESpec("l_least", 1, 1, 32, 32, Q4, SILU),
    wl.MoESpec("l_least_shared", 2, 1, 32, 32, Q8, GELU, 32, I4),
    wl.MoESpec("l_i4_odd_units", 200, 8, 2080, 736, I4, SILU),
]


def router(spec, seed):
    return wl.normal_f32(seed, wl.stream_id(f"{spec.name}/R"), spec.n_experts * spec.hidden,
                         std=0.02).view(spec.n_experts, spec.hidden)


def check(spec, x, R, y, idx, w, seed=0, tol=TOL, what=""):
    logits = om.router_logits(R.numpy(), x.numpy())
    ridx, rw = om.router_topk(logits, spec.top_k)
    # the inputs' own choice is clear of the fp32 sums' error, so the indices have to agree
    order = -np.sort(-logits, axis=1)[:, :spec.top_k + 1]
    gap = np.min(order[:, :-1] - order[:, 1:]) if order.shape[1] > 1 else 1.0
    assert gap > 1e-6 * np.max(np.abs(logits)), "choose another seed: two logits are too close"
    assert np.array_equal(idx.cpu().numpy(), ridx), what
    assert_close(w, rw, tol=1e-5, what=what)
    ref = om.moe_layer(oracle_layer(spec, seed), x.numpy(), ridx, rw)
    assert_close(y, ref, tol=tol, what=what)


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("spec", SMALL, ids=lambda s: s.name)
def test_small_layers(spec, tokens):
    need_gpu()
    T = wl.build_moe_layer(spec, 0, 0, device="cuda")
    L = device_layer(T)
    x, R = wl.moe_tokens(spec, 0, tokens), router(spec, 0)
    ws = bqg.moe_layer_workspace(L, tokens)
    y, idx, w = bqg.moe_layer(L, R.cuda(), x.cuda(), workspace=ws)
    torch.cuda.synchronize()
    assert bqg.bqg_device_errors() == 0
    check(spec, x, R, y, idx, w, what=f"{spec.name} T={tokens}")
    assert not ws[:bqg.MOE_LAYER_STATE_BYTES].any()
    y2, idx2, w2 = bqg.moe_layer(L, R.cuda(), x.cuda(), workspace=ws)
    assert torch.equal(y, y2) and torch.equal(idx, idx2) and torch.equal(w, w2)  # deterministic


FULL = [
    (wl.GEMMA_MOE, 1), (wl.GEMMA_MOE, 8),
    (wl.MoESpec("l_glm24", 24, 8, 6144, 2048, I4, SILU), 1), (wl.MoESpec("l_glm24", 24, 8, 6144, 2048, I4, SILU), 3),
    (wl.MoESpec("l_glm24", 24, 8, 6144, 2048, I4, SILU), 8),
    (wl.MoESpec("l_widest", 3, 2, 7168, 7168, Q8, GELU, 7168, Q4), 2),
    (wl.MoESpec("l_widest_i2", 4, 2, 7168, 3584, I2, SILU, 7168, Q8), 7),
]


@pytest.mark.parametrize("spec,tokens", FULL, ids=lambda v: v.name if hasattr(v, "name") else str(v))
def test_full_width_layers(spec, tokens):
    need_gpu()
    T = wl.build_moe_layer(spec, 0, 0, device="cuda")
    x, R = wl.moe_tokens(spec, 0, tokens), router(spec, 0)
    y, idx, w = bqg.moe_layer(device_layer(T), R.cuda(), x.cuda())
    torch.cuda.synchronize()
    assert bqg.bqg_device_errors() == 0
    check(spec, x, R, y, idx, w, what=f"{spec.name} T={tokens}")


def test_ties_go_to_the_lower_index():
    need_gpu()
    spec = wl.MoESpec("l_ties", 70, 8, 64, 32, Q4, SILU)
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    x = wl.moe_tokens(spec, 0, 4)
    y, idx, w = bqg.moe_layer(L, torch.zeros(70, 64, device="cuda"), x.cuda())
    assert idx.cpu().tolist() == [list(range(8))] * 4
    assert torch.allclose(w, torch.full_like(w, 1 / 8), rtol=2 ** -22, atol=0)
    ridx = np.tile(np.arange(8, dtype=np.int32), (4, 1))
    ref = om.moe_layer(oracle_layer(spec, 0), x.numpy(), ridx, np.full((4, 8), 1 / 8))
    assert_close(y, ref, tol=TOL)
    R = router(spec, 0)
    R[69], R[3], R[40] = R[11], R[11], R[11]   # equal rows: equal logits, bit for bit
    _, idx, _ = bqg.moe_layer(L, R.cuda(), x.cuda())
    lg = om.router_logits(R.numpy(), x.numpy())
    assert np.array_equal(idx.cpu().numpy(), om.topk_select(lg, 8))


def test_zero_and_nonfinite_tokens_stay_apart():
    """A token of zeros gives zeros; a token with a NaN or an Inf gives NaN in its own row only."""
    need_gpu()
    for spec in (SMALL[0], SMALL[2], SMALL[5]):
        L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
        x, R = wl.moe_tokens(spec, 0, 5), router(spec, 0)
        x[1] = 0
        x[2, 5] = float("nan")
        x[3, 0] = float("inf")
        y, idx, w = bqg.moe_layer(L, R.cuda(), x.cuda())
        torch.cuda.synchronize()
        assert bqg.bqg_device_errors() == 0
        assert (y[1] == 0).all() and idx[1].cpu().tolist() == list(range(spec.top_k))
        assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
        assert ((idx >= 0) & (idx < spec.n_experts)).all()
        keep = [0, 4]
        check(spec, x[keep], R, y[keep], idx[keep], w[keep])


def test_agrees_with_the_separate_calls():
    """The layer as router, top-k and moe_forward, at that path's own bound."""
    need_gpu()
    for spec in SMALL[:5]:
        L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
        x, R = wl.moe_tokens(spec, 0, 6).cuda(), router(spec, 0).cuda()
        idx, w = bqg.moe_router_topk(bqg.moe_router_logits(R, x), spec.top_k)
        y = bqg.moe_forward(L.with_path(bqg.MOE_PATH_CUDA_CORES), x, idx, w)
        y2, idx2, w2 = bqg.moe_layer(L, R, x)
        assert torch.equal(idx, idx2)
        assert_close(w2, w.cpu().numpy(), tol=1e-6)
        assert_close(y2, y.cpu().numpy(), tol=1e-4 + TOL)


def test_workspace_of_more_tokens_and_in_turn():
    """One workspace for calls of several token counts, one after another, and larger buffers whose
    rest stays as it was."""
    need_gpu()
    spec = SMALL[4]
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    R = router(spec, 0)
    sizes = [bqg.moe_layer_workspace_size(L, t) for t in range(1, 9)]
    ws = bqg.moe_layer_workspace(L, 8)
    assert ws.numel() == max(sizes)
    for tokens in (8, 1, 3, 8, 2, 1):
        x = wl.moe_tokens(spec, 0, tokens)
        y = torch.full((9, spec.hidden), -5.0, device="cuda")
        idx = torch.full((9, spec.top_k), -5, dtype=torch.int32, device="cuda")
        w = torch.full((9, spec.top_k), -5.0, device="cuda")
        bqg.moe_layer(L, R.cuda(), x.cuda(), y, idx, w, ws)
        check(spec, x, R, y[:tokens], idx[:tokens], w[:tokens])
        assert (y[tokens:] == -5).all() and (idx[tokens:] == -5).all() and (w[tokens:] == -5).all()


def test_routing_outputs_are_optional():
    need_gpu()
    spec = SMALL[0]
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    x, R = wl.moe_tokens(spec, 0, 2).cuda(), router(spec, 0).cuda()
    want, _, _ = bqg.moe_layer(L, R, x)
    y, ws = torch.empty_like(want), bqg.moe_layer_workspace(L, 2)
    s = torch.cuda.current_stream().cuda_stream
    assert bqg.lib().moe_layer(ctypes.addressof(L.c), R.data_ptr(), x.data_ptr(), y.data_ptr(), None, None, 2,
                               ws.data_ptr(), ws.numel(), s) == 0
    assert torch.equal(y, want)


def test_graphs_and_streams():
    """Captured and replayed with new inputs; two graphs that share a workspace, replayed in turn;
    calls on several streams at once, each with its own workspace."""
    need_gpu()
    spec = SMALL[3]
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    R = router(spec, 0).cuda()
    ws = bqg.moe_layer_workspace(L, 8)
    made = []
    for tokens in (1, 6):
        x = wl.moe_tokens(spec, 0, tokens).cuda()
        out = bqg.moe_layer(L, R, x, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                bqg.moe_layer(L, R, x, *out, workspace=ws)
        made.append((g, x, out))
    for seed in (1, 2, 3):
        for g, x, out in made:
            x.copy_(wl.moe_tokens(spec, seed, x.shape[0]))
            out[0].zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, x, out in made:
            check(spec, x.cpu(), R.cpu(), *out)
    jobs = []
    for i in range(4):
        x = wl.moe_tokens(spec, 10 + i, 1 + 2 * i).cuda()
        jobs.append((x, bqg.moe_layer_workspace(L, 1 + 2 * i), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs = []
        for x, w8, st in jobs:
            with torch.cuda.stream(st):
                outs.append(bqg.moe_layer(L, R, x, workspace=w8))
    torch.cuda.synchronize()
    assert bqg.bqg_device_errors() == 0
    for (x, _, _), out in zip(jobs, outs):
        check(spec, x.cpu(), R.cpu(), *out)


def test_decode_step_of_a_layer():
    """The operators as a decode step uses them: the token batch through an int8 projection, then the
    routed layer on its output, in one graph."""
    need_gpu()
    from oracle import i8 as oi
    spec = wl.MoESpec("l_step", 16, 4, 512, 256, Q4, SILU, 128, Q8)
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    R = router(spec, 0)
    g = torch.Generator().manual_seed(3)
    a = torch.randn(4, 300, generator=g).bfloat16()
    wq, sw = bqg.quantize_rows_i8(torch.randn(512, 300, generator=g).cuda() * 0.06)
    a_dev, ws = a.cuda(), bqg.moe_layer_workspace(L, 4)
    Xq = torch.empty(4, 304, dtype=torch.int8, device="cuda")[:, :300]
    sx = torch.empty(4, device="cuda")
    h = torch.empty(4, 512, device="cuda")
    y, idx, w = torch.empty_like(h), torch.empty(4, 4, dtype=torch.int32, device="cuda"), torch.empty(4, 4, device="cuda")

    def step():
        bqg.quantize_rows_i8(a_dev, Xq, sx)
        bqg.qgemm_i8(Xq, sx, wq, sw, Y=h)
        bqg.moe_layer(L, R_dev, h, y, idx, w, ws)
    R_dev = R.cuda()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    q, s = oi.quantize_rows(a.float().numpy())
    ref_h = oi.product(q, s, wq.cpu().numpy(), sw.cpu().numpy())
    assert np.array_equal(Xq.cpu().numpy(), q)
    assert np.max(np.abs(h.cpu().numpy() - ref_h) / np.abs(ref_h)) <= 3 * 2.0 ** -24 * 1.01
    check(spec, h.cpu(), R, y, idx, w)


def test_binding_refusals():
    need_gpu()
    spec = SMALL[0]
    L = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda"))
    x, R = wl.moe_tokens(spec, 0, 2).cuda(), router(spec, 0).cuda()
    with pytest.raises(bqg.BQGError):                      # more tokens than the call takes
        bqg.moe_layer(L, R, torch.zeros(9, spec.hidden, device="cuda"))
    with pytest.raises(ValueError):
        bqg.moe_layer_workspace(L, 9)
    with pytest.raises(ValueError):
        bqg.moe_layer(L, R[:-1], x)
    with pytest.raises(ValueError):
        bqg.moe_layer(L, R, x[:, :100].contiguous())
    with pytest.raises(TypeError):
        bqg.moe_layer(L, R, x.double())
    with pytest.raises(ValueError):
        bqg.moe_layer(L, R, x, y=torch.empty(1, spec.hidden, device="cuda"))
    with pytest.raises(ValueError):
        bqg.moe_layer(L, R, x, w=torch.empty(1, spec.top_k, device="cuda"))
    with pytest.raises(bqg.BQGError):                      # a workspace of fewer tokens
        bqg.moe_layer(L, R, x, workspace=bqg.moe_layer_workspace(L, 1))
