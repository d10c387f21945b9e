"""GPU: whole verify steps and decode chains on the 4-bit cache and with a
sliding window: store, attention, acceptance and compaction together."""
import math

import pytest
import torch

import ext_reference as R
from oracle import medusa_oracle as O
from medusa_head_speculative_02_b200 import api
from medusa_head_speculative_02_b200.decode import DecodeLoop
from medusa_head_speculative_02_b200.step import PackedVerifyStep, VerifyStep
from medusa_head_speculative_02_b200.synthetic import MedusaConfig

pytestmark = pytest.mark.gpu
BF = MedusaConfig("packed_small", "bf16", B=3, d=512, V=1000, K=4, s=3, N=33, Hq=4, Hkv=2, dh=128,
                  L_lo=100, L_hi=301)
F32 = MedusaConfig("packed_tiny", "f32", B=2, d=256, V=1024, K=4, s=3, N=16, Hq=4, Hkv=4, dh=64,
                   L_lo=17, L_hi=130)
ONE = MedusaConfig("packed_token", "bf16", B=2, d=256, V=512, K=1, s=1, N=1, Hq=8, Hkv=2, dh=128,
                   L_lo=40, L_hi=90)


def _weights(c):
    return "fp32" if c.dtype == "f32" else "fp16"


def _store_reference(arrs, st, L):
    """The step's stored rows and compaction on CPU copies of the cache arrays."""
    c = st.cfg
    for x, i in ((st.tree_k, 0), (st.tree_v, 2)):
        codes, scale, zero = R.encode(x)
        for b in range(c.B):
            for n in range(c.N):
                arrs[i][b, :, L[b] + n] = codes[b, n]
                arrs[i + 1][b, :, L[b] + n, 0] = scale[b, n].to(torch.bfloat16)
                arrs[i + 1][b, :, L[b] + n, 1] = zero[b, n].to(torch.bfloat16)


def _compact_reference(arrs, L, alen, nodes):
    for t in arrs:
        for b in range(len(L)):
            for j in range(1, alen[b] + 1):
                t[b, :, L[b] + j] = t[b, :, L[b] + nodes[b][j]]


@pytest.mark.parametrize("cfg", [BF, F32, ONE], ids=lambda c: c.name)
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_packed_chain_matches_the_definitions(cfg, window, sinks):
    """Three chained steps: cache contents bit for bit, attention within its
    bound, acceptance and lengths those of the step on the bf16/fp32 cache."""
    steps = 3
    loop = DecodeLoop(cfg, "cuda", seed=3, max_steps=steps, packed=True, window=window, sinks=sinks)
    st, c = loop.st, loop.cfg
    ref_step = VerifyStep(c, "cuda", 3)   # same heads, tree tokens and verify logits
    arrs = [t.clone().cpu() for t in (st.cache.k_codes, st.cache.k_par, st.cache.v_codes, st.cache.v_par)]
    plan = O.tree_plan(c.K, c.s, c.N)
    for _ in range(steps):
        L = st.x["prefix_len"].tolist()
        ref_step.x["prefix_len"].copy_(st.x["prefix_len"])
        ref_step.x["root_tok"].copy_(st.x["root_tok"])
        loop.step()
        ref_step.run()
        _store_reference(arrs, st, L)
        k, v = (R.decode(arrs[i], arrs[i + 1]).cuda() for i in (0, 2))
        ref = R.attention(st.x["q"], k, v, L, plan, st.scale, window, sinks)
        R.assert_close(st.attn_out, *ref, c.torch_dtype, _weights(c))
        for name in ("tree_tok", "tree_pos", "accept_len", "accept_nodes", "next_tok", "new_len"):
            assert torch.equal(getattr(st, name), getattr(ref_step, name)), name
        _compact_reference(arrs, L, st.accept_len.tolist(), st.accept_nodes.tolist())
        got = (st.cache.k_codes, st.cache.k_par, st.cache.v_codes, st.cache.v_par)
        for g, w in zip(got, arrs):
            assert torch.equal(g.cpu(), w)
        assert st.x["prefix_len"].tolist() == [l + 1 + a for l, a in zip(L, st.accept_len.tolist())]
    assert api.device_status() == 0


@pytest.mark.parametrize("packed", [True, False])
def test_graph_replay_equals_eager_chain(packed):
    steps = 3
    loop = DecodeLoop(BF, "cuda", seed=5, max_steps=steps + 1, packed=packed, window=90, sinks=2)
    outs = []
    for _ in range(steps):
        loop.step()
        outs.append((loop.st.attn_out.clone(), loop.st.new_len.clone(), loop.st.next_tok.clone()))
    final = {k: v.clone() for k, v in loop.st.state().items()}
    loop.reset()
    loop.capture()
    for i in range(steps):
        loop.step()
        for got, want in zip((loop.st.attn_out, loop.st.new_len, loop.st.next_tok), outs[i]):
            assert torch.equal(got, want)
    for k, v in loop.st.state().items():
        assert torch.equal(v, final[k]), k


def test_windowed_step_on_the_bf16_cache():
    st = VerifyStep(BF, "cuda", 7, window=50, sinks=3)
    st.run()
    L = st.x["prefix_len"].tolist()
    # compaction moved rows after attention: compare with the inputs drawn again
    from medusa_head_speculative_02_b200.synthetic import gen_attention_inputs
    x = gen_attention_inputs(BF, "cuda", 7)
    ref = R.attention(x["q"], x["k_cache"].double().transpose(1, 2),
                      x["v_cache"].double().transpose(1, 2), L, O.tree_plan(BF.K, BF.s, BF.N),
                      1 / math.sqrt(BF.dh), 50, 3)
    R.assert_close(st.attn_out, *ref, torch.bfloat16, "bf16")


def test_launch_counts_and_layers():
    """launches_per_step counts the store too; compaction over a cache with a
    layer axis moves every layer's rows as the single call does."""
    st = PackedVerifyStep(BF, "cuda", 1)
    plain = VerifyStep(BF, "cuda", 1)
    assert st.launches_per_step() in (plain.launches_per_step(), plain.launches_per_step() + 1,
                                      plain.launches_per_step() + 2)
    st.run()
    many = api.PackedCache.empty(BF.B, BF.Hkv, st.Lcap, BF.dh, "cuda", layers=2)
    for i in range(2):
        api.medusa_kv_pack(st.tree_k, st.tree_v, many.layer(i), st.x["prefix_len"])
    one = many.layer(1)
    one = api.PackedCache(*(t.clone() for t in (one.k_codes, one.k_par, one.v_codes, one.v_par)))
    args = (st.x["prefix_len"], st.accept_len, st.accept_nodes, BF.K)
    api.medusa_kv_compact_packed(many, *args)
    api.medusa_kv_compact_packed(one, *args)
    for i in range(2):
        got = many.layer(i)
        for a, b in zip((got.k_codes, got.k_par, got.v_codes, got.v_par),
                        (one.k_codes, one.k_par, one.v_codes, one.v_par)):
            assert torch.equal(a, b)
