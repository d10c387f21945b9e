"""GPU: every call on a 4-bit cache refuses one whose tensors no longer have
the sizes it was made with."""
import pytest
import torch

from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
B, HKV, LCAP, DH, N = 2, 2, 64, 128, 8


@pytest.mark.parametrize("name", ["k_codes", "k_par", "v_codes", "v_par"])
@pytest.mark.parametrize("how", ["resized", "smaller", "strided"])
def test_a_changed_cache_is_refused(name, how):
    cache = api.PackedCache.empty(B, HKV, LCAP, DH)
    t, dev = getattr(cache, name), "cuda"
    if how == "resized":
        t.resize_(B, HKV, LCAP // 2, t.shape[-1])
    elif how == "smaller":
        t.data = t[:, :, :LCAP - 4].clone()
    else:
        t.data = t.new_zeros(B, LCAP, HKV, t.shape[-1]).transpose(1, 2)
    tree = api.Tree(3, 2, N)
    q = torch.randn(B, N, 4, DH, device=dev, dtype=torch.bfloat16)
    new = torch.randn(B, N, HKV, DH, device=dev, dtype=torch.bfloat16)
    length = torch.full((B,), 20, dtype=torch.int32, device=dev)
    path = torch.zeros(B, 4, dtype=torch.int32, device=dev)
    for call in (lambda: api.medusa_tree_attention_packed(q, cache, length, tree, 0.1),
                 lambda: api.medusa_kv_pack(new, new, cache, length),
                 lambda: api.medusa_kv_unpack(cache, length, 3),
                 lambda: api.medusa_kv_compact_packed(cache, length, length, path, 3)):
        with pytest.raises(ValueError, match=name):
            call()
    torch.cuda.synchronize()
    assert api.device_status() == 0
