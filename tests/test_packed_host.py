"""CPU: argument checks of the 4-bit cache and windowed attention calls, made
before any CUDA call, and the 64-bit forms the GPU tests compare with."""
import ctypes as C
import math

import pytest
import torch

import ext_reference as R
from oracle import medusa_oracle as O
from medusa_head_speculative_02_b200 import _lib as L
from medusa_head_speculative_02_b200 import api

P = C.c_void_p(256)
ODD = C.c_void_p(264)


def _pack(B=1, T=4, H=2, dh=128, Lcap=8, dt=L.BF16, k=P, start=P, kc=P, vp=P):
    return L.lib().medusa_kv_pack(k, P, dt, start, None, B, T, H, dh, Lcap, kc, P, P, vp, None)


def _unpack(B=1, T=4, H=2, dh=128, Lcap=8, dt=L.BF16, out=P, kc=P):
    return L.lib().medusa_kv_unpack(kc, P, P, P, P, None, B, T, H, dh, Lcap, dt, P, out, None)


def _compact(B=1, H=2, dh=128, Lcap=8, K=4, layers=1, kc=P, alen=P, new_len=None):
    return L.lib().medusa_kv_compact_packed(kc, P, P, P, layers, P, alen, P, B, H, dh, Lcap, K,
                                            new_len, None)


@pytest.mark.parametrize("fn", [_pack, _unpack])
def test_store_and_read_refusals(fn):
    assert fn(dt=7) == L.ERR_INVALID_ARG
    assert fn(B=-1) == L.ERR_INVALID_ARG
    assert fn(T=-1) == L.ERR_INVALID_ARG
    assert fn(H=0) == L.ERR_INVALID_ARG
    assert fn(Lcap=0) == L.ERR_INVALID_ARG
    assert fn(dh=96) == L.ERR_UNSUPPORTED
    assert fn(Lcap=10) == L.ERR_UNSUPPORTED
    assert b"multiple of 4" in L.lib().medusa_last_error()
    assert fn(kc=None) == L.ERR_INVALID_ARG
    assert fn(kc=ODD) == L.ERR_INVALID_ARG
    assert b"aligned" in L.lib().medusa_last_error()
    assert fn(B=0) == L.OK and fn(T=0) == L.OK   # nothing to do


def test_more_store_refusals():
    assert _pack(k=ODD) == L.ERR_INVALID_ARG
    assert _pack(start=None) == L.ERR_INVALID_ARG
    assert _pack(vp=None) == L.ERR_INVALID_ARG
    assert _unpack(out=ODD) == L.ERR_INVALID_ARG


def test_compact_refusals():
    assert _compact(K=9) == L.ERR_INVALID_ARG
    assert _compact(K=-1) == L.ERR_INVALID_ARG
    assert _compact(layers=-1) == L.ERR_INVALID_ARG
    assert _compact(dh=32) == L.ERR_UNSUPPORTED
    assert _compact(Lcap=6) == L.ERR_UNSUPPORTED
    assert _compact(alen=None) == L.ERR_INVALID_ARG
    assert _compact(kc=ODD) == L.ERR_INVALID_ARG
    assert _compact(new_len=P) == L.ERR_INVALID_ARG       # the lengths themselves
    assert b"new_len" in L.lib().medusa_last_error()
    assert _compact(alen=ODD, new_len=ODD) == L.ERR_INVALID_ARG
    assert _compact(B=0) == L.OK and _compact(layers=0) == L.OK


def test_attention_calls_need_a_tree():
    lib = L.lib()
    assert lib.medusa_tree_attention_window(P, P, P, P, None, 1, 4, 4, 128, 64, 0.1, L.BF16, 8, 0,
                                            P, P, 1, None) == L.ERR_INVALID_ARG
    assert lib.medusa_tree_attention_packed(P, P, P, P, P, P, None, 1, 4, 4, 128, 64, 0.1, L.BF16,
                                            8, 0, P, P, 1, None) == L.ERR_INVALID_ARG
    assert lib.medusa_tree_attention_packed_workspace_size(None, 1, 4, 4, 128, 64, L.BF16, 0, 0) == 0
    assert lib.medusa_tree_attention_window_workspace_size(None, 1, 4, 4, 128, 64, L.BF16, 0, 0) == 0


def test_binding_refuses_bad_tensors():
    c = torch.zeros(1, 2, 8, 64, dtype=torch.uint8)
    p = torch.zeros(1, 2, 8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.PackedCache(c, p, c, p)
    with pytest.raises(TypeError):
        api.PackedCache([1], p, c, p)


def test_reference_row_format():
    x = torch.tensor([[0.0, 1.0, -0.5, 14.5, 2.5, 0.49, 7.0, -0.5]])
    codes, scale, zero = R.encode(x)
    assert float(scale) == 1.0 and float(zero) == 0.0   # -(-0.5) / 1 is a tie: to even
    c = [int(codes[0, 0]) & 15, int(codes[0, 0]) >> 4, int(codes[0, 1]) & 15, int(codes[0, 1]) >> 4]
    assert c == [0, 1, 0, 14]                          # 14.5 is a tie: to even
    par = torch.stack([scale, zero], -1).to(torch.bfloat16)
    assert R.decode(codes, par)[0].tolist() == [0, 1, 0, 14, 2, 0, 7, 0]
    _, scale, _ = R.encode(torch.tensor([[1.0, math.nan]]))
    assert math.isnan(float(scale))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 2), (50, 9)])
def test_reference_visibility(window, sinks):
    """The vectorised rule equals the rule written out, a node always sees
    itself, and window 1 without sinks leaves only that."""
    depth, anc = R.tree_masks(O.tree_plan(4, 3, 16))
    for Lb in (0, 1, 7, 20):
        v = R.visible_fast(depth, anc, Lb, window, sinks)
        assert torch.equal(v, R.visible(depth, anc, Lb, window, sinks))
        assert bool(v[torch.arange(16), Lb + torch.arange(16)].all())
        if window == 1 and sinks == 0:
            assert int(v.sum()) == 16
