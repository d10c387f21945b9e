"""Failure detection of the tcgen05 4-bit attention kernels, whose source has
status words of its own: a bounded wait there that runs out is reported, kept
until it is cleared, and leaves the context usable."""
import pytest
import torch

from medusa_head_speculative_02_b200 import _lib as L
from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu


def test_a_wait_that_runs_out_there_is_reported_and_cleared():
    torch.cuda.synchronize()
    assert api.device_status(clear=True) == L.OK
    api.selftest_wait_timeout(50, packed=True)
    assert api.device_status(clear=False) == L.ERR_TIMEOUT
    assert api.device_status(clear=True) == L.ERR_TIMEOUT   # read, then cleared
    assert api.device_status(clear=False) == L.OK
    # each source's word alone, and both
    for packed in (False, True, None):
        for p in (False, True) if packed is None else (packed,):
            api.selftest_wait_timeout(5, packed=p)
        assert api.device_status(clear=True) == L.ERR_TIMEOUT
        assert api.device_status(clear=True) == L.OK


def test_the_4_bit_attention_runs_after_it():
    tree = api.Tree(5, 10, 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(1, n, 2, 128, generator=g, device="cuda").bfloat16() for n in (64, 300))
    cache = api.PackedCache.empty(1, 2, 364, 128)
    length = torch.tensor([236], dtype=torch.int32, device="cuda")
    api.medusa_kv_pack(k, k, cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
    want = api.medusa_tree_attention_packed(q, cache, length, tree, 0.09).clone()
    api.selftest_wait_timeout(5, packed=True)
    assert torch.equal(api.medusa_tree_attention_packed(q, cache, length, tree, 0.09), want)
    assert api.device_status(clear=True) == L.ERR_TIMEOUT


def test_limit_out_of_range_is_rejected():
    for bad in (0, -5, 2001):
        with pytest.raises(L.MedusaError, match="limit_ms"):
            api.selftest_wait_timeout(bad, packed=True)
