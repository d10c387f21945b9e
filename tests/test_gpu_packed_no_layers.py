"""GPU: compaction of a 4-bit cache without layers still answers the lengths."""
import pytest
import torch

from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu


def test_lengths_without_layers():
    cache = api.PackedCache.empty(3, 2, 16, 64, layers=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    length, alen = torch.tensor([5, 0, 7], **i32), torch.tensor([2, 0, 9], **i32)
    nodes, new = torch.zeros(3, 5, **i32), torch.full((3,), -7, **i32)
    api.medusa_kv_compact_packed(cache, length, alen, nodes, 4, new_len=new)
    assert new.tolist() == [8, 1, -1]            # (an accepted length past K: -1)
    assert api.medusa_kv_compact_packed(cache, length, alen, nodes, 4).tolist() == [8, 1, -1]
