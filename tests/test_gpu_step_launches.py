"""GPU: launches_per_step is the number of kernels that a captured step holds,
for the bf16/fp32 and the 4-bit cache, with and without a window."""
import pytest
import torch

from medusa_head_speculative_02_b200.step import MultiLayerStep, PackedVerifyStep, VerifyStep
from medusa_head_speculative_02_b200.synthetic import MedusaConfig

pytestmark = pytest.mark.gpu
CONFIGS = [
    MedusaConfig("bf16", "bf16", B=3, d=512, V=1000, K=4, s=3, N=33, Hq=4, Hkv=2, dh=128,
                 L_lo=100, L_hi=301),
    MedusaConfig("f32", "f32", B=2, d=256, V=1024, K=4, s=3, N=16, Hq=4, Hkv=4, dh=64,
                 L_lo=17, L_hi=130),
    MedusaConfig("token", "bf16", B=2, d=256, V=512, K=1, s=1, N=1, Hq=8, Hkv=2, dh=128,
                 L_lo=40, L_hi=90),
    MedusaConfig("batch40", "bf16", B=40, d=512, V=1000, K=2, s=3, N=5, Hq=2, Hkv=1, dh=128,
                 L_lo=10, L_hi=40, accept="both"),
    MedusaConfig("rows_long", "bf16", B=1, d=256, V=512, K=5, s=10, N=64, Hq=2, Hkv=2, dh=128,
                 L_lo=9000, L_hi=9001),
]


def _kernels(fn) -> int:
    from cuda.bindings import runtime as rt
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        fn()
    raw = g.raw_cuda_graph()
    err, _, n = rt.cudaGraphGetNodes(raw)
    err, nodes, n = rt.cudaGraphGetNodes(raw, n)
    assert err == rt.cudaError_t.cudaSuccess
    types = [rt.cudaGraphNodeGetType(x)[1] for x in nodes[:n]]
    return sum(t == rt.cudaGraphNodeType.cudaGraphNodeTypeKernel for t in types)


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4), (5000, 0)])
@pytest.mark.parametrize("step", [VerifyStep, PackedVerifyStep], ids=["plain", "packed"])
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: c.name)
def test_launches_are_those_of_a_captured_step(cfg, step, window, sinks):
    st = step(cfg, "cuda", 1, window, sinks)
    assert st.launches_per_step() == _kernels(st.run)
    if step is PackedVerifyStep:
        assert _kernels(st.store) == 1 and _kernels(st.compact) == 1


@pytest.mark.parametrize("cfg", CONFIGS[:2], ids=lambda c: c.name)
def test_launches_of_a_step_through_layers(cfg):
    st = MultiLayerStep(cfg, 3, "cuda", 1)
    assert st.launches_per_step() == _kernels(st.run)
