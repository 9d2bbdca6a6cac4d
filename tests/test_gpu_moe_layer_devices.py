"""moe_layer refuses a layer any of whose tensors is not on the device of x, before a launch: the kernel would
read an address of another memory."""
import pytest

import block_quant_gemv_b200 as bqg
from synth import workloads as wl
from tests.test_gpu_moe_layer import SMALL, router
from tests.util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", range(6))
def test_a_matrix_on_the_host(which):
    need_gpu()
    spec = SMALL[0]
    T = wl.build_moe_layer(spec, 0, 0, device="cuda")
    mats = [T.gate, T.up, T.down, *T.shared]
    mats[which] = mats[which].cpu()
    L = bqg.MoELayer(spec.n_experts, spec.top_k, spec.hidden, spec.inter, spec.expert_fmt, spec.act, *mats[:3],
                     T.gate_stride, T.up_stride, T.down_stride, (spec.shared_fmt, spec.shared_inter, *mats[3:]))
    with pytest.raises(ValueError, match="one device"):
        bqg.moe_layer(L, router(spec, 0).cuda(), wl.moe_tokens(spec, 0, 2).cuda())
