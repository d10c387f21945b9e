"""GPU: kernels launched before their predecessor has finished read nothing
ahead of it.  Every buffer that a step's kernels hand on is overwritten with
a value no step produces before each run; a kernel that read its input before
the kernel ahead had written it would turn that value into another result
(the fp32 step's compaction did: it lost new_len in 265 of 300 runs)."""
import pytest
import torch

from medusa_head_speculative_02_b200 import api
from medusa_head_speculative_02_b200.step import PackedVerifyStep, VerifyStep
from medusa_head_speculative_02_b200.synthetic import MedusaConfig

pytestmark = pytest.mark.gpu
CONFIGS = [
    MedusaConfig("f32", "f32", B=2, d=256, V=1024, K=4, s=3, N=16, Hq=4, Hkv=4, dh=64, L_lo=17,
                 L_hi=130),
    MedusaConfig("bf16", "bf16", B=3, d=512, V=1000, K=4, s=3, N=33, Hq=4, Hkv=2, dh=128, L_lo=100,
                 L_hi=301, accept="both"),
    MedusaConfig("typical", "bf16", B=3, d=512, V=1000, K=4, s=3, N=12, Hq=4, Hkv=4, dh=64, L_lo=100,
                 L_hi=301, accept="typical"),
]
NAMES = ("topk_idx", "tree_tok", "tree_pos", "accept_len", "accept_nodes", "next_tok", "new_len")


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: c.name)
@pytest.mark.parametrize("kind", [VerifyStep, PackedVerifyStep])
def test_steps_from_poisoned_buffers(cfg, kind):
    st = kind(cfg, "cuda", 3)
    start = {k: v.clone() for k, v in st.state().items()}

    def run():
        for k, v in st.state().items():
            v.copy_(start[k])
        for k in NAMES:
            getattr(st, k).fill_(-7)
        st.topk_val.fill_(float("nan"))
        st.attn_out.fill_(float("nan"))
        for ws in (st.ws_heads, st.ws_attn, st.ws_acc):
            ws.fill_(255)
        st.run()
        torch.cuda.synchronize()
        out = {k: getattr(st, k).clone() for k in NAMES + ("attn_out",)}
        out.update({k: v.clone() for k, v in st.state().items()})
        return out

    first = run()
    assert int(first["new_len"].min()) > 0
    for i in range(40):
        again = run()
        for k, v in first.items():
            assert torch.equal(again[k], v), (i, k)


def test_store_and_sampling_follow_their_producers():
    """Lengths and nodes written by one call are read by the next, on one
    stream with nothing between."""
    cfg = CONFIGS[0]
    st = PackedVerifyStep(cfg, "cuda", 4)
    st.run()
    torch.cuda.synchronize()
    want_tok = api.medusa_sample_next(st.vlogits, st.accept_len, st.accept_nodes, 0.9, 5, 1).clone()
    cache = api.PackedCache.empty(cfg.B, cfg.Hkv, st.Lcap + 16, cfg.dh, "cuda")
    api.medusa_kv_pack(st.tree_k, st.tree_v, cache, st.new_len)
    want = cache.k_codes.clone()
    tok = torch.empty_like(want_tok)
    for _ in range(40):
        for t in (st.accept_len, st.accept_nodes, st.new_len, tok):
            t.fill_(-7)
        cache.k_codes.zero_()
        st.accept()
        api.medusa_sample_next(st.vlogits, st.accept_len, st.accept_nodes, 0.9, 5, 1, out=tok)
        st.compact()
        api.medusa_kv_pack(st.tree_k, st.tree_v, cache, st.new_len)
        torch.cuda.synchronize()
        assert torch.equal(tok, want_tok) and torch.equal(cache.k_codes, want)
