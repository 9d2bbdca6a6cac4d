"""GPU parity of int8 row quantization where many rows take 64 or 128 threads each: q and the scale are
compared bit for bit with the oracle, on rows that meet exact ties and the neighbourhood of borders."""
import numpy as np
import pytest
import torch

import block_quant_gemv_b200 as bqg
from oracle import i8 as oi
from tests.test_gpu_i8 import TYPES, rows
from tests.util import need_gpu

pytestmark = pytest.mark.gpu


def check(X):
    q, s = bqg.quantize_rows_i8(X)
    ref_q, ref_s = oi.quantize_rows(X.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.int32), ref_s.view(np.int32))
    assert np.array_equal(q.cpu().numpy(), ref_q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r,k,pitch", [(593, 1025, None), (600, 1999, 2003), (700, 2048, 2056), (593, 2049, None),
                                       (640, 4096, None), (601, 4095, 4097), (593, 4097, None), (9, 1024, None)])
def test_many_rows_bit_exact(r, k, pitch, dtype):
    need_gpu()
    check(rows(r + k, r, k, dtype, pitch))


@pytest.mark.parametrize("k", [600, 1500, 3500])
def test_borders_and_their_neighbours(k):
    """Quotients at n + 1/2 (scale 1), and one fp32 step to either side of it under other scales."""
    need_gpu()
    g = torch.Generator().manual_seed(k)
    half = torch.randint(-126, 126, (600, k), generator=g).float() + 0.5
    half[:, 0] = 127
    scale = torch.exp(torch.randn(600, 1, generator=g) * 8)
    scale[:100] = 1
    x = half * scale
    step = torch.randint(-1, 2, (600, k), generator=g).to(torch.int32)
    step[:, 0] = 0
    x = (x.view(torch.int32) + step).view(torch.float32)
    check(x.cuda())
