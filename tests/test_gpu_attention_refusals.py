"""Refusals of the windowed and the 4-bit attention calls, all made on the
host, and their calls without sequences."""
import pytest
import torch

from medusa_head_speculative_02_b200 import _lib as L
from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
B, HQ, HKV, DH, LCAP = 2, 4, 2, 128, 64


@pytest.fixture(scope="module")
def tree():
    return api.Tree(3, 2, 8)


def _inputs(n=8, b=B, hq=HQ, dh=DH, lcap=LCAP, dtype=torch.bfloat16):
    dev = "cuda"
    q = torch.randn(b, n, hq, dh, device=dev, dtype=dtype)
    k = torch.randn(b, lcap, HKV, dh, device=dev, dtype=dtype)
    v = torch.randn(b, lcap, HKV, dh, device=dev, dtype=dtype)
    length = torch.full((b,), 20, dtype=torch.int32, device=dev)
    cache = api.PackedCache.empty(b, HKV, lcap, dh, dev)
    return q, k, v, length, cache


def _both(tree, q, k, v, length, cache, scale=0.1, window=8, sinks=0, **kw):
    return (lambda: api.medusa_tree_attention_window(q, k, v, length, tree, scale, window, sinks, **kw),
            lambda: api.medusa_tree_attention_packed(q, cache, length, tree, scale, window, sinks, **kw))


def _refused(calls, exc, match=None):
    for c in calls:
        with pytest.raises(exc, match=match):
            c()


def test_arguments(tree):
    x = _inputs()
    _refused(_both(tree, *x, window=-1), ValueError, "window")
    _refused(_both(tree, *x, sinks=-1), ValueError, "window")
    _refused(_both(tree, *x, window=2**32), ValueError, "window")  # no silent window 0
    _refused(_both(tree, *x, sinks=2**31), ValueError, "window")
    for s in (0.0, -1.0, float("nan"), float("inf")):
        _refused(_both(tree, *x, scale=s), L.MedusaError, "scale")


def test_shapes_and_types(tree):
    q, k, v, length, cache = _inputs()
    _refused(_both(tree, q[:, :7].contiguous(), k, v, length, cache), ValueError)
    _refused(_both(tree, q[:, :, :3].contiguous(), k, v, length, cache), L.MedusaError, "Hq")
    _refused(_both(tree, q.transpose(1, 2), k, v, length, cache), ValueError)
    _refused(_both(tree, q.half(), k, v, length, cache), TypeError)
    _refused(_both(tree, q, k, v, length.long(), cache), TypeError)
    _refused(_both(tree, q, k, v, length[:1], cache), ValueError)
    _refused(_both(tree, q, k, v, length.cpu(), cache), ValueError)
    _refused(_both(tree, q.cpu(), k, v, length, cache), ValueError)
    _refused(_both(tree, q, k, v, length, cache, out=q.float()), TypeError)
    _refused(_both(tree, q, k, v, length, cache, out=q[:1]), ValueError)
    _refused(_both(tree, q, k.float(), v, length, cache)[:1], TypeError)
    _refused(_both(tree, q, k, v[:, :32], length, cache)[:1], ValueError)
    with pytest.raises(ValueError, match="layer"):
        api.medusa_tree_attention_packed(q, api.PackedCache.empty(B, HKV, LCAP, DH, layers=2),
                                         length, tree, 0.1)
    with pytest.raises(AttributeError):
        cache.k_codes = cache.v_codes


def test_limits(tree):
    _refused(_both(tree, *_inputs(dh=96)), L.MedusaError, "dh")
    q, k, v, length, _ = _inputs(lcap=62)
    odd = api.PackedCache.empty(B, HKV, 62, DH)
    with pytest.raises(L.MedusaError, match="multiple of 4"):
        api.medusa_tree_attention_packed(q, odd, length, tree, 0.1)
    api.medusa_tree_attention_window(q, k, v, length, tree, 0.1, 8)  # any Lcap here
    _refused(_both(tree, *_inputs(lcap=4)), L.MedusaError, "Lcap")


def test_alignment(tree):
    q, k, v, length, cache = _inputs()
    off = torch.empty(q.numel() + 4, dtype=q.dtype, device="cuda")[4:].view(q.shape)
    _refused(_both(tree, off, k, v, length, cache), L.MedusaError, "aligned")
    _refused(_both(tree, q, k, v, length, cache, out=off), L.MedusaError, "aligned")
    offk = torch.empty(k.numel() + 4, dtype=k.dtype, device="cuda")[4:].view(k.shape)
    _refused(_both(tree, q, offk, v, length, cache)[:1], L.MedusaError, "aligned")
    codes = torch.zeros(cache.k_codes.numel() + 4, dtype=torch.uint8, device="cuda")[4:]
    bad = api.PackedCache(codes.view(cache.k_codes.shape), cache.k_par, cache.v_codes, cache.v_par)
    _refused(_both(tree, q, k, v, length, bad)[1:], L.MedusaError, "aligned")


def test_workspace(tree):
    """A workspace that is too small: the C call refuses it, the binding takes
    one of its own."""
    q, k, v, length, cache = _inputs(dtype=torch.float32)  # SIMT: always partial rows
    need = api.attention_packed_workspace_size(tree, B, HQ, HKV, DH, LCAP, torch.float32, 8, 0)
    assert need > 0
    out = torch.empty_like(q)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for ptr, n in ((ws.data_ptr(), need - 1), (None, need), (ws.data_ptr() + 8, need)):
        rc = L.lib().medusa_tree_attention_packed(
            q.data_ptr(), *cache._ptrs, length.data_ptr(), tree.handle, B, HQ, HKV, DH, LCAP, 0.1,
            L.F32, 8, 0, out.data_ptr(), ptr, n, None)
        assert rc == L.ERR_INVALID_ARG
    a = api.medusa_tree_attention_packed(q, cache, length, tree, 0.1, 8, ws=ws[:16])
    assert torch.equal(a, api.medusa_tree_attention_packed(q, cache, length, tree, 0.1, 8, ws=ws))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_sequences(tree, dtype):
    q, k, v, length, cache = _inputs(b=0, dtype=dtype)
    for c in _both(tree, q, k, v, length, cache):
        assert c().shape == q.shape
    zero = torch.zeros(0, dtype=torch.int32, device="cuda")
    new = torch.zeros(0, 3, HKV, DH, dtype=dtype, device="cuda")
    api.medusa_kv_pack(new, new, cache, zero)
    assert api.medusa_kv_unpack(cache, zero, 5, dtype)[0].shape == (0, 5, HKV, DH)
    path = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert api.medusa_kv_compact_packed(cache, zero, zero, path, 3).numel() == 0
    torch.cuda.synchronize()
    assert api.device_status() == 0


def test_sequences_outside_the_cache(tree):
    """A negative length, and one whose tree does not fit: rows of zeros, the
    others untouched by it."""
    q, k, v, length, cache = _inputs(b=3)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    api.medusa_kv_pack(k, v, cache, zero)
    good = [c() for c in _both(tree, q, k, v, length, cache)]
    length = torch.tensor([-1, 20, LCAP - 7], dtype=torch.int32, device="cuda")
    for c, g in zip(_both(tree, q, k, v, length, cache), good):
        o = c()
        assert torch.equal(o[1], g[1])
        assert not o[0].any() and not o[2].any()


def test_cache_follows_its_tensors(tree):
    """A tensor of the cache given other memory: the calls read the new one."""
    q, k, v, length, cache = _inputs()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    api.medusa_kv_pack(k, v, cache, zero)
    want = api.medusa_tree_attention_packed(q, cache, length, tree, 0.1)
    cache.k_codes.data, old = cache.k_codes.clone(), cache.k_codes.data
    old.zero_()
    assert torch.equal(api.medusa_tree_attention_packed(q, cache, length, tree, 0.1), want)
