"""The scaled int8 product's roundings, bit for bit: fp32(sum), times the token's scale, times the channel's,
plus the bias, each rounded to fp32, then the output type, on every path (one to eight tokens, tiles of
one CTA, tiles that share k, CTA pairs)."""
import numpy as np
import pytest
import torch

import block_quant_gemv_b200 as bqg
from tests.test_gpu_i8 import TYPES, int8_rows
from tests.util import need_gpu

pytestmark = pytest.mark.gpu
SHAPES = [(1, 512, 200), (2, 48, 77), (3, 500, 64), (8, 640, 333), (16, 128, 130), (40, 500, 64), (24, 4096, 512),
          (300, 64, 301), (1200, 96, 700), (3000, 64, 3000)]


def inputs(tokens, k, n):
    q, w = int8_rows(tokens + k, tokens, k), int8_rows(tokens + k + 1, n, k)
    g = torch.Generator().manual_seed(n)
    # values of either sign, a bias about as large as the sums: where a fused step would show
    sx, sw, bias = (torch.rand(m, generator=g) * 2 - 1 for m in (tokens, n, n))
    return q, sx, w, sw, bias * (k ** 0.5 * 2000)


@pytest.mark.parametrize("tokens,k,n", SHAPES)
@pytest.mark.parametrize("biased", [False, True])
def test_each_step_is_rounded(tokens, k, n, biased):
    need_gpu()
    q, sx, w, sw, bias = inputs(tokens, k, n)
    v = (q.double() @ w.double().T).cpu().numpy().astype(np.float32) * sx.numpy()[:, None] * sw.numpy()
    if biased:
        v = v + bias.numpy()
    for out in TYPES:
        y = bqg.qgemm_i8(q, sx.cuda(), w, sw.cuda(), out, bias.cuda() if biased else None)
        assert torch.equal(y.cpu(), torch.from_numpy(v).to(out))
