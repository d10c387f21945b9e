"""CPU: the work that a verify step reports for its attention call."""
import pytest
import torch

import ext_reference as R
from oracle import medusa_oracle as O
from medusa_head_speculative_02_b200 import kernel_bench as KB
from medusa_head_speculative_02_b200.step import VerifyStep
from medusa_head_speculative_02_b200.synthetic import MedusaConfig

CFG = MedusaConfig("host", "bf16", B=3, d=512, V=1000, K=4, s=3, N=16, Hq=4, Hkv=2, dh=128,
                   L_lo=10, L_hi=301)
WINDOWS = [(0, 0), (0, 9), (1, 0), (1, 5), (3, 2), (50, 0), (50, 9), (50, 400), (1000, 4)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_visible_prefix_counts_the_slots_some_node_sees(window, sinks):
    depth, anc = R.tree_masks(O.tree_plan(CFG.K, CFG.s, CFG.N))
    for L in (0, 1, 2, 7, 49, 50, 51, 200):
        seen = R.visible_fast(depth, anc, L, window, sinks).any(0)
        assert KB.visible_prefix(L, window, sinks) == int(seen[:L].sum())


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_attention_work_follows_the_window(window, sinks):
    st = object.__new__(VerifyStep)  # (its buffers need a GPU)
    Ls = [10, 300, 77]
    st.cfg, st.window, st.sinks = CFG, window, sinks
    st.x = {"prefix_len": torch.tensor(Ls, dtype=torch.int32)}
    n = sum(KB.visible_prefix(L, window, sinks) for L in Ls)
    assert st.attention_bytes() == (2 * (n + 48) * 2 * 128 + 2 * 48 * 4 * 128) * 2
    assert st.attention_flops() == 4 * 4 * 16 * (n + 48) * 128
    if window == 0:
        assert n == sum(Ls)
