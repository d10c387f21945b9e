"""GPU: tree attention over the 4-bit cache and with a sliding window, against
the formula in 64 bits, with the bounds derived in ext_reference."""
import math

import pytest
import torch

import ext_reference as R
from canary import Guarded, GuardedWorkspace
from oracle import medusa_oracle as O
from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _lcap(Ls, N, spare=0):
    return (max(Ls) + N + spare + 3) // 4 * 4


def _packed_inputs(B, tree, Hq, Hkv, dh, Ls, dtype, seed=0, spare=5):
    K, s, N = tree
    g = torch.Generator(device=DEV).manual_seed(seed * 977 + B * 31 + N + Hq)
    Lcap = _lcap(Ls, N, spare)
    q = torch.randn(B, N, Hq, dh, generator=g, device=DEV).to(dtype)
    c = api.PackedCache.empty(B, Hkv, Lcap, dh, DEV)
    for x in (c.k_codes, c.v_codes):
        x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV, dtype=torch.int16))
    for p in (c.k_par, c.v_par):
        # scales spread over a factor of 8, zeros over the code range
        p[..., 0] = torch.rand(p.shape[:-1], generator=g, device=DEV).mul_(3).exp2_().mul_(0.08)
        p[..., 1] = torch.randint(4, 12, p.shape[:-1], generator=g, device=DEV).float()
    L = torch.tensor(Ls, dtype=torch.int32, device=DEV)
    return q, c, L, Lcap


def _values(c):
    return R.decode(c.k_codes, c.k_par), R.decode(c.v_codes, c.v_par)


def _weights(dtype, dh, G, N, packed=True):
    """Rounding of the kernel that takes this shape (ext_reference.C_P)."""
    if dtype == F32 or dh == 64 or (not packed and 128 % G):
        return "fp32"
    if not packed:
        return "bf16"
    return "fp16v" if N * G > 128 else "fp16"


# (B, tree (K, s, N), Hq, Hkv, dh, prefix lengths, dtype)
SHAPES = [
    (1, (1, 1, 1), 1, 1, 128, [0], BF),                 # one token, nothing cached
    (1, (1, 1, 1), 8, 1, 128, [1], BF),
    (2, (1, 1, 1), 32, 8, 128, [700, 129], BF),         # single tokens, GQA
    (1, (5, 10, 64), 4, 4, 128, [128], BF),
    (2, (5, 10, 64), 4, 4, 128, [300, 129], BF),
    (1, (5, 10, 64), 32, 32, 128, [2048], BF),          # 7B-shaped
    (3, (5, 10, 63), 6, 2, 128, [0, 257, 1000], BF),    # 189 rows
    (2, (4, 3, 17), 14, 2, 128, [511, 40], BF),         # group of 7
    (2, (5, 8, 128), 8, 2, 128, [1200, 640], BF),       # 512 rows
    (1, (5, 3, 256), 3, 3, 128, [900], BF),
    (1, (5, 3, 200), 2, 2, 128, [60], BF),
    (4, (2, 4, 21), 5, 5, 128, [1, 127, 0, 383], BF),
    (1, (4, 3, 16), 4, 4, 64, [128], F32),              # tiny
    (2, (5, 3, 40), 6, 3, 64, [77, 300], BF),
    (2, (4, 3, 30), 8, 2, 128, [150, 3], F32),
    (1, (5, 8, 100), 4, 2, 64, [500], F32),
]
WINDOWS = [(0, 0), (1, 0), (100, 4), (64, 130), (5000, 16)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("B,tree,Hq,Hkv,dh,Ls,dtype", SHAPES)
def test_packed_matches_the_formula(B, tree, Hq, Hkv, dh, Ls, dtype, window, sinks):
    q, c, L, _ = _packed_inputs(B, tree, Hq, Hkv, dh, Ls, dtype)
    scale = 1 / math.sqrt(dh)
    got = api.medusa_tree_attention_packed(q, c, L, api.Tree(*tree), scale, window, sinks)
    ref = R.attention(q, *_values(c), Ls, O.tree_plan(*tree), scale, window, sinks)
    R.assert_close(got, *ref, dtype, _weights(dtype, dh, Hq // Hkv, tree[2]))
    assert api.device_status() == 0


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("B,tree,Hq,Hkv,dh,Ls,dtype", SHAPES)
def test_window_matches_the_formula(B, tree, Hq, Hkv, dh, Ls, dtype, window, sinks):
    K, s, N = tree
    g = torch.Generator(device=DEV).manual_seed(B * 31 + N + Hq)
    Lcap = max(Ls) + N + 3
    q = torch.randn(B, N, Hq, dh, generator=g, device=DEV).to(dtype)
    k = torch.randn(B, Lcap, Hkv, dh, generator=g, device=DEV).to(dtype)
    v = torch.randn(B, Lcap, Hkv, dh, generator=g, device=DEV).to(dtype)
    L = torch.tensor(Ls, dtype=torch.int32, device=DEV)
    scale = 1 / math.sqrt(dh)
    t = api.Tree(*tree)
    got = api.medusa_tree_attention_window(q, k, v, L, t, scale, window, sinks)
    ref = R.attention(q, k.double().transpose(1, 2), v.double().transpose(1, 2), Ls,
                      O.tree_plan(*tree), scale, window, sinks)
    R.assert_close(got, *ref, dtype, _weights(dtype, dh, Hq // Hkv, N, packed=False))
    assert api.device_status() == 0


@pytest.mark.parametrize("tree,Hq", [((5, 10, 64), 2), ((1, 1, 1), 8), ((4, 3, 5), 6),
                                     ((4, 3, 9), 6), ((5, 10, 50), 4), ((5, 3, 200), 2)])
@pytest.mark.parametrize("scale_q", [1e-3, 40.0])
def test_packed_growing_maxima(scale_q, tree, Hq):
    """Scores that grow along the prefix (the running maximum moves in every
    tile) and value scales that grow by 2^40 over it, in every kernel."""
    q, c, L, Lcap = _packed_inputs(1, tree, Hq, 2, 128, [1500], BF, spare=0)
    q = (q.float() * scale_q).to(BF)
    ramp = torch.linspace(0, 1, Lcap, device=DEV)
    c.k_par[..., 0] *= (1 + 6 * ramp).to(BF)
    c.v_par[..., 0] *= (40 * (ramp - 0.5)).exp2().to(BF)
    scale = 1 / math.sqrt(128)
    for w, s in ((0, 0), (300, 7)):
        got = api.medusa_tree_attention_packed(q, c, L, api.Tree(*tree), scale, w, s)
        ref = R.attention(q, *_values(c), [1500], O.tree_plan(*tree), scale, w, s)
        R.assert_close(got, *ref, BF, _weights(BF, 128, Hq // 2, tree[2]))


@pytest.mark.parametrize("B,tree,Hq,Hkv,dh,Ls,dtype", [SHAPES[2], SHAPES[4], SHAPES[6], SHAPES[8],
                                                       SHAPES[13], SHAPES[14]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_slots_no_node_sees_may_hold_anything(B, tree, Hq, Hkv, dh, Ls, dtype, window, sinks):
    """Unused capacity and slots that have left every window: NaN scales there
    change no bit of the output.  The same for a bf16/fp32 cache."""
    N = tree[2]
    q, c, L, Lcap = _packed_inputs(B, tree, Hq, Hkv, dh, Ls, dtype)
    t, plan, scale = api.Tree(*tree), O.tree_plan(*tree), 1 / math.sqrt(dh)
    depth, anc = R.tree_masks(plan)
    k, v = (x.transpose(1, 2).to(dtype).contiguous() for x in _values(c))
    clean = api.medusa_tree_attention_packed(q, c, L, t, scale, window, sinks).clone()
    cleanw = api.medusa_tree_attention_window(q, k, v, L, t, scale, window, sinks).clone()
    for b, Lb in enumerate(Ls):
        dead = torch.ones(Lcap, dtype=torch.bool)
        dead[:Lb + N] = ~R.visible_fast(depth, anc, Lb, window, sinks).any(0)
        dead = dead.to(DEV)
        for par in (c.k_par, c.v_par):
            par[b, :, dead] = math.nan
        for x in (k, v):
            x[b, dead] = math.nan
    assert torch.equal(api.medusa_tree_attention_packed(q, c, L, t, scale, window, sinks), clean)
    assert torch.equal(api.medusa_tree_attention_window(q, k, v, L, t, scale, window, sinks), cleanw)


@pytest.mark.parametrize("dh,dtype,tree", [(128, BF, (4, 3, 16)), (64, BF, (4, 3, 16)),
                                           (128, F32, (4, 3, 16)), (128, BF, (4, 3, 6)),
                                           (128, BF, (4, 3, 60)), (128, BF, (5, 3, 110))])
def test_a_visible_nan_row_reaches_exactly_its_nodes(dh, dtype, tree):
    Ls = [70, 200]
    q, c, L, _ = _packed_inputs(2, tree, 4, 2, dh, Ls, dtype)
    depth, anc = R.tree_masks(O.tree_plan(*tree))
    c.k_par[0, 1, 70 + 3] = math.nan         # node 3's key of kv-head 1
    c.v_par[1, 0, 200 + 2] = math.nan        # node 2's value of kv-head 0
    out = api.medusa_tree_attention_packed(q, c, L, api.Tree(*tree), 0.1).isnan()
    want = torch.zeros_like(out)
    want[0, :, 2:] |= anc[:, 3].to(DEV)[:, None, None]
    want[1, :, :2] |= anc[:, 2].to(DEV)[:, None, None]
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype,dh", [(BF, 128), (F32, 64)])
def test_sequences_that_do_not_fit_and_canaries(dtype, dh):
    """L_b < 0 or L_b + N > Lcap: rows of zeros, the others untouched by it;
    no write outside the output and a workspace of exactly the asked size."""
    tree, Hq, Hkv = (5, 10, 33), 6, 2
    Ls = [100, 500, 40]
    q, c, L, Lcap = _packed_inputs(3, tree, Hq, Hkv, dh, Ls, dtype, spare=0)
    t, scale = api.Tree(*tree), 1 / math.sqrt(dh)
    k, v = (x.transpose(1, 2).to(dtype).contiguous() for x in _values(c))
    for bad in (-1, Lcap - 32, 2 ** 31 - 1, -2 ** 31):
        L2 = L.clone()
        L2[1] = bad
        for w, s in ((0, 0), (77, 5), (2 ** 31 - 1, 2 ** 31 - 1)):
            for packed in (True, False):
                out = Guarded(q.shape, dtype, DEV)
                size = (api.attention_packed_workspace_size if packed
                        else api.attention_window_workspace_size)(t, 3, Hq, Hkv, dh, Lcap, dtype, w, s)
                ws = GuardedWorkspace(max(size, 1), DEV)
                if packed:
                    api.medusa_tree_attention_packed(q, c, L2, t, scale, w, s, out=out.t, ws=ws.t)
                else:
                    api.medusa_tree_attention_window(q, k, v, L2, t, scale, w, s, out=out.t, ws=ws.t)
                assert out.intact() and ws.intact()
                assert out.t[1].abs().max() == 0
                ref = R.attention(q, *(_values(c) if packed else (x.double().transpose(1, 2) for x in (k, v))),
                                  [100, bad, 40], O.tree_plan(*tree), scale, w, s)
                R.assert_close(out.t, *ref, dtype, _weights(dtype, dh, Hq // Hkv, tree[2], packed))


def test_unwindowed_call_equals_tree_attention():
    """window = 0 is medusa_tree_attention, bit for bit (bf16, dh = 128)."""
    tree = (5, 10, 64)
    q, c, L, _ = _packed_inputs(2, tree, 4, 4, 128, [300, 1290], BF)
    k, v = (x.transpose(1, 2).to(BF).contiguous() for x in _values(c))
    t = api.Tree(*tree)
    a = api.medusa_tree_attention(q, k, v, L, t, 0.088)
    b = api.medusa_tree_attention_window(q, k, v, L, t, 0.088, 0)
    assert torch.equal(a, b)


@pytest.mark.parametrize("window", [0, 200])
def test_repeatable_and_captured_on_another_stream(window):
    tree, Ls = (5, 10, 64), [900, 333]
    q, c, L, Lcap = _packed_inputs(2, tree, 8, 4, 128, Ls, BF)
    k, v = (x.transpose(1, 2).to(BF).contiguous() for x in _values(c))
    t, scale = api.Tree(*tree), 0.09
    call = {True: lambda: api.medusa_tree_attention_packed(q, c, L, t, scale, window, 4),
            False: lambda: api.medusa_tree_attention_window(q, k, v, L, t, scale, window, 4)}
    for packed, fn in call.items():
        first = fn().clone()
        for _ in range(3):
            assert torch.equal(fn(), first)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = fn()
        s.synchronize()
        assert torch.equal(other, first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = fn()
        L.copy_(torch.tensor([41, 700], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref = R.attention(q, *(_values(c) if packed else (x.double().transpose(1, 2) for x in (k, v))),
                          [41, 700], O.tree_plan(*tree), scale, window, 4)
        R.assert_close(o, *ref, BF, "fp16" if packed else "bf16")
        L.copy_(torch.tensor(Ls, dtype=torch.int32))


@pytest.mark.parametrize("N,Hq", [(20, 8), (64, 8), (40, 24)])  # 20, 64 and 120 rows per kv-head
@pytest.mark.parametrize("Ls,fused", [([0, 1900, 130], True), ([5, 7900, 3000], False)])
def test_chunk_merge_in_a_cluster_and_in_the_workspace(N, Hq, Ls, fused):
    """Key chunks that merge in a cluster (no workspace) and, more than 8 of
    them, in the workspace: sequences shorter than the chunks are many, and one
    that does not fit."""
    tree, Hkv = (5, 10, N), 8 if fused else 2
    Hq = Hq * Hkv // 8
    q, c, L, Lcap = _packed_inputs(3, tree, Hq, Hkv, 128, Ls, BF, spare=0)
    t = api.Tree(*tree)
    size = api.attention_packed_workspace_size(t, 3, Hq, Hkv, 128, Lcap, BF)
    assert (size == 0) == fused
    for bad in (None, 2 ** 31 - 1):
        L2, Lb = L.clone(), list(Ls)
        if bad is not None:
            L2[1], Lb[1] = bad, bad
        out, ws = Guarded(q.shape, BF, DEV), GuardedWorkspace(max(size, 1), DEV)
        api.medusa_tree_attention_packed(q, c, L2, t, 0.088, out=out.t, ws=ws.t)
        assert out.intact() and ws.intact()
        ref = R.attention(q, *_values(c), Lb, O.tree_plan(*tree), 0.088, 0, 0)
        R.assert_close(out.t, *ref, BF, "fp16")
        first = out.t.clone()
        for _ in range(3):
            assert torch.equal(api.medusa_tree_attention_packed(q, c, L2, t, 0.088), first)
    assert api.device_status() == 0
