"""The first call of a process may be one that is captured into a graph: nothing that a call does once (kernel
attributes, the number of clusters that run at once) disturbs the capture."""
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from tests.util import need_gpu

pytestmark = pytest.mark.gpu

INT8 = """
import torch, block_quant_gemv_b200 as bqg
from tests.test_gpu_i8 import int8_rows
shapes = [(1, 512, 300), (16, 4096, 4352), (40, 500, 300), (300, 200, 500), (2600, 64, 2600)]
jobs = []
for t, k, n in shapes:
    jobs.append((int8_rows(1, t, k), torch.ones(t, device="cuda"), int8_rows(2, n, k), torch.ones(n, device="cuda"),
                 torch.zeros(t, n, device="cuda")))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for q, sx, w, sw, y in jobs:
        bqg.qgemm_i8(q, sx, w, sw, Y=y)
    q8, s8 = bqg.quantize_rows_i8(jobs[3][4])
for _ in range(2):
    for job in jobs:
        job[4].zero_()
    g.replay()
    torch.cuda.synchronize()
    for q, sx, w, sw, y in jobs:
        assert torch.equal(y, (q.double() @ w.double().T).float())
    assert torch.equal(s8, (jobs[3][4].abs().amax(1).double() / 127).float())
assert bqg.bqg_device_errors() == 0
"""
LAYER = """
import torch, block_quant_gemv_b200 as bqg
from synth import workloads as wl
from tests.moe_util import device_layer
from tests.test_gpu_moe_layer import SMALL, check, router
spec = SMALL[4]
L, R, x = device_layer(wl.build_moe_layer(spec, 0, 0, device="cuda")), router(spec, 0), wl.moe_tokens(spec, 0, 3)
Rd, xd = R.cuda(), x.cuda()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, idx, w = bqg.moe_layer(L, Rd, xd)  # its own workspace, zeroed in the graph
for _ in range(3):
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(spec, x, R, y, idx, w)
assert bqg.bqg_device_errors() == 0
"""


@pytest.mark.parametrize("program", [INT8, LAYER], ids=["int8", "moe_layer"])
def test_captured_first(program):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
