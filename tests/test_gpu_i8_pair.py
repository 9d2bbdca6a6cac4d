"""GPU parity of the scaled int8 product at the sizes that CTA pairs compute (256 channels x 256 tokens
a tile, many tiles): against exact sums, and bit for bit against the same rows in smaller calls."""
import pytest
import torch

import block_quant_gemv_b200 as bqg
from tests.test_gpu_i8 import TYPES, int8_rows
from tests.util import need_gpu

pytestmark = pytest.mark.gpu
SHAPES = [(3000, 200, 3001), (4096, 128, 2560), (4097, 1000, 2561), (2305, 31, 4700), (5000, 16, 2300)]


@pytest.mark.parametrize("tokens,k,n", SHAPES)
def test_exact_sums(tokens, k, n):
    """Scales of 1: the outputs are the int32 sums, below 2^24 and so exact in fp32."""
    need_gpu()
    q, w = int8_rows(tokens + k, tokens, k), int8_rows(tokens + k + 1, n, k)
    one = torch.ones(max(tokens, n), device="cuda")
    y = bqg.qgemm_i8(q, one[:tokens], w, one[:n], torch.float32)
    assert torch.equal(y.double(), q.double() @ w.double().T)
    assert bqg.bqg_device_errors() == 0


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("pitch", [0, 3])
def test_same_bits_as_smaller_calls(out, pitch):
    """Scales, a bias and a row pitch; other numbers of tokens take the other paths."""
    need_gpu()
    tokens, k, n = 4097, 300, 2500
    q, w = int8_rows(5, tokens, k), int8_rows(6, n, k)
    g = torch.Generator().manual_seed(7)
    sx, sw, bias = (torch.rand(m, generator=g).cuda() + 0.5 for m in (tokens, n, n))
    buf = torch.full((tokens + 2, n + pitch), -7.0, dtype=out, device="cuda")
    y = bqg.qgemm_i8(q, sx, w, sw, bias=bias, Y=buf[:tokens, :n])
    for a, b in ((0, 6), (250, 270), (256, 400), (1000, 1300), (4000, 4097)):
        assert torch.equal(bqg.qgemm_i8(q[a:b], sx[a:b], w, sw, out, bias), y[a:b]), (a, b)
    assert (buf[tokens:] == -7).all() and (buf[:, n:] == -7).all()


def test_in_a_graph_and_on_two_streams():
    need_gpu()
    jobs = []
    for i in range(2):
        q, w = int8_rows(30 + i, 3000, 256), int8_rows(40 + i, 3001, 256)
        jobs.append((q, w, torch.ones(3001, device="cuda"), torch.empty(3000, 3001, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, w, one, y, st in jobs:
            with torch.cuda.stream(st):
                bqg.qgemm_i8(q, one, w, one, Y=y)
    torch.cuda.synchronize()
    for q, w, one, y, _ in jobs:
        assert torch.equal(y.double(), q.double() @ w.double().T)
    q, w, one, y, _ = jobs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xq, sx = bqg.quantize_rows_i8(q.float())
        bqg.qgemm_i8(xq, sx, w, one, Y=y)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    xq, sx = bqg.quantize_rows_i8(q.float())
    assert torch.equal(y, bqg.qgemm_i8(xq, sx, w, one, torch.float32))
    assert bqg.bqg_device_errors() == 0


@pytest.mark.parametrize("tokens,k,n", [(25000, 64, 100), (20003, 200, 128)])
def test_many_tokens_few_channels(tokens, k, n):
    """128 x 256 tiles of single CTAs: one row of channels, more tiles than CTA pairs."""
    need_gpu()
    q, w = int8_rows(1, tokens, k), int8_rows(2, n, k)
    one = torch.ones(tokens, device="cuda")
    y = bqg.qgemm_i8(q, one, w, one[:n], torch.float32)
    assert torch.equal(y.double(), q.double() @ w.double().T)
    assert bqg.bqg_device_errors() == 0
