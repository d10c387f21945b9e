"""4-bit cache whose byte offsets pass 32 bits: what is stored, read, attended to
and moved far behind equals the same in a small cache, bit for bit."""
import pytest
import torch

from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, DH = 9, 128
FAR = 8 * 1024 * 1024          # slots per kv-head: 4.8 GB of codes each for K and V
NEAR = 512
SHIFT = FAR - NEAR             # a multiple of 128: the same places within key tiles


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype,G,N", [
    (torch.bfloat16, 1, 8),      # few query rows
    (torch.bfloat16, 4, 16),     # keys as the MMA's rows
    (torch.bfloat16, 4, 64),     # two query tiles
    (torch.float32, 2, 8),       # SIMT
])
def test_far_slots(dtype, G, N):
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free device memory")
    g = torch.Generator(device=DEV).manual_seed(3)
    k = torch.randn(1, NEAR - 56, H, DH, device=DEV, generator=g).to(dtype)
    v = torch.randn(1, NEAR - 56, H, DH, device=DEV, generator=g).to(dtype)
    q = torch.randn(1, N, G * H, DH, device=DEV, generator=g).to(dtype)
    tree = api.Tree(4, 4, N)
    L = NEAR - 56 - N
    alen, nodes = _i32(2), torch.tensor([[0, 2, 5, -1, -1]], dtype=torch.int32, device=DEV)
    got = []
    for cap, off in ((NEAR, 0), (FAR, SHIFT)):
        cache = api.PackedCache.empty(1, H, cap, DH, DEV)
        api.medusa_kv_pack(k, v, cache, _i32(off))
        out = api.medusa_tree_attention_packed(q, cache, _i32(off + L), tree, 0.1, window=200)
        new_len = api.medusa_kv_compact_packed(cache, _i32(off + L), alen, nodes, 4)
        back = api.medusa_kv_unpack(cache, _i32(off), NEAR - 56, dtype)
        got.append((out, new_len - off, *back))
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert not torch.equal(got[0][2], k)  # 4-bit values, not the stored ones
    assert got[0][0].isfinite().all() and got[0][0].abs().sum() > 0
