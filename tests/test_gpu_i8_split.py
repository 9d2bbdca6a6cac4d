"""GPU parity of the scaled int8 product where a cluster of CTAs shares a tile's k (few tiles, long rows):
against exact sums, and bit for bit against the same rows as single tokens."""
import pytest
import torch

import block_quant_gemv_b200 as bqg
from tests.test_gpu_i8 import TYPES, int8_rows
from tests.util import need_gpu

pytestmark = pytest.mark.gpu
SHAPES = [(9, 4096, 130), (16, 8192, 100), (12, 65536, 140), (24, 4096, 4096), (24, 2060, 1200), (30, 8190, 1000),
          (64, 8192, 300), (100, 2051, 1000), (128, 8192, 128), (129, 3500, 250), (256, 4096, 1000), (300, 6000, 500)]


@pytest.mark.parametrize("tokens,k,n", SHAPES)
def test_exact_sums(tokens, k, n):
    """Scales of 1: the outputs are the int32 sums, rounded once to fp32."""
    need_gpu()
    q, w = int8_rows(tokens + k, tokens, k), int8_rows(tokens + k + 1, n, k)
    one = torch.ones(max(tokens, n), device="cuda")
    for _ in range(2):
        y = bqg.qgemm_i8(q, one[:tokens], w, one[:n], torch.float32)
        assert torch.equal(y, (q.double() @ w.double().T).float())
    assert bqg.bqg_device_errors() == 0


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("tokens,k,n,pitch", [(24, 4096, 1001, 1004), (100, 2051, 1000, 1000), (60, 8192, 301, 304),
                                              (17, 5000, 129, 129)])
def test_same_bits_as_single_tokens(tokens, k, n, pitch, out):
    need_gpu()
    q, w = int8_rows(5, tokens, k), int8_rows(6, n, k)
    g = torch.Generator().manual_seed(7)
    sx, sw, bias = (torch.rand(m, generator=g).cuda() + 0.5 for m in (tokens, n, n))
    buf = torch.full((tokens + 2, pitch), -7.0, dtype=out, device="cuda")
    bqg.qgemm_i8(q, sx, w, sw, bias=bias, Y=buf[:tokens, :n])
    for a in range(0, tokens, 5):
        b = min(a + 5, tokens)
        assert torch.equal(bqg.qgemm_i8(q[a:b], sx[a:b], w, sw, out, bias), buf[a:b, :n]), (a, b)
    assert (buf[tokens:] == -7).all() and (buf[:, n:] == -7).all()


def test_in_a_graph_and_on_two_streams():
    need_gpu()
    jobs = []
    for i in range(3):
        q, w = int8_rows(30 + i, 24, 4096), int8_rows(40 + i, 2000, 4096)
        jobs.append((q, w, torch.ones(2000, device="cuda"), torch.empty(24, 2000, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, w, one, y, st in jobs:
            with torch.cuda.stream(st):
                bqg.qgemm_i8(q, one[:24], w, one, Y=y)
    torch.cuda.synchronize()
    for q, w, one, y, _ in jobs:
        assert torch.equal(y, (q.double() @ w.double().T).float())
    q, w, one, y, _ = jobs[0]
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            bqg.qgemm_i8(q, one[:24], w, one, Y=y)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and bqg.bqg_device_errors() == 0
