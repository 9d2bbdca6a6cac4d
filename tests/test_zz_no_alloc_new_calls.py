"""quantize_rows_i8, qgemm_i8 and moe_layer allocate nothing when the caller hands them their outputs (and
moe_layer its workspace): neither through torch nor from the device behind it, at first use of a size or later."""
import pytest
import torch

import block_quant_gemv_b200 as bqg
from synth import workloads as wl
from tests.moe_util import device_layer
from tests.test_gpu_i8 import int8_rows, rows
from tests.test_gpu_moe_layer import SMALL, router
from tests.util import need_gpu

pytestmark = pytest.mark.gpu


def allocations():
    torch.cuda.synchronize()
    return torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]


def test_int8_calls():
    need_gpu()
    jobs = []
    for tokens, k, n in ((1, 512, 300), (40, 500, 300), (24, 4096, 512), (2600, 64, 2600)):
        jobs.append((rows(tokens, tokens, k, torch.bfloat16), int8_rows(1, tokens, k), torch.empty(tokens, device="cuda"),
                     int8_rows(2, n, k), torch.rand(n, device="cuda"), torch.empty(tokens, n, device="cuda")))

    def run():
        for X, Xq, sx, W, sw, Y in jobs:
            bqg.quantize_rows_i8(X, Xq, sx)
            bqg.qgemm_i8(Xq, sx, W, sw, Y=Y)
    run()  # the kernels' code is loaded when they first run
    before = allocations()
    for _ in range(3):
        run()
    assert allocations() == before


def test_moe_layer():
    need_gpu()
    jobs = []
    for spec in SMALL[:4]:
        L, R = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda")), router(spec, 0).cuda()
        for tokens in (1, 8):
            x = wl.moe_tokens(spec, 0, tokens).cuda()
            ws = bqg.moe_layer_workspace(L, tokens)
            jobs.append((L, R, x, *bqg.moe_layer(L, R, x, workspace=ws), ws))
    before = allocations()
    for _ in range(3):
        for job in jobs:
            bqg.moe_layer(*job)
    assert allocations() == before
