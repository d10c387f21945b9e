"""GPU: a cached row with scale NaN reaches the nodes that see it however
small its weight: a key 200 nats above all others leaves it a softmax weight
of exactly 0, and 0 x NaN is NaN."""
import pytest
import torch

from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

# (tree (K, s, N), query heads per kv-head, dh, dtype)
KERNELS = {
    "rows8": ((4, 3, 5), 1, 128, BF),
    "rows16": ((4, 3, 5), 3, 128, BF),
    "keys32": ((4, 3, 9), 3, 128, BF),
    "keys64": ((5, 10, 50), 1, 128, BF),
    "keys128": ((5, 10, 50), 2, 128, BF),
    "pair": ((5, 3, 200), 1, 128, BF),
    "simt64": ((4, 3, 30), 2, 64, BF),
    "simt_f32": ((5, 3, 40), 1, 128, F32),
}
# (kv-heads, prefix): one chunk, chunks that merge in a cluster (bf16, dh = 128,
# 17 to 128 rows), chunks in the workspace
CHUNKS = {"one": (160, 700), "few": (4, 700), "many": (2, 7900)}


def _call(kernel, chunks, nan, big, which):
    """Output of queries of ones over K rows near 0, one of them ~211 nats above
    the others at slot `big`; scale NaN in K and / or V at slot `nan`."""
    tree, G, dh, dtype = KERNELS[kernel]
    Hkv, L = CHUNKS[chunks]
    N = tree[2]
    g = torch.Generator(device=DEV).manual_seed(N + G + L)
    c = api.PackedCache.empty(1, Hkv, (L + N + 3) // 4 * 4, dh, DEV)
    for x in (c.k_codes, c.v_codes):
        x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV, dtype=torch.int16))
    for p in (c.k_par, c.v_par):
        p[..., 0] = 0.05
        p[..., 1] = 8
    c.k_codes[:, :, big] = 255
    c.k_par[:, :, big, 0] = 211.0 / (0.1 * dh * 15)
    c.k_par[:, :, big, 1] = 0
    if "k" in which:
        c.k_par[:, :, nan, 0] = float("nan")
    if "v" in which:
        c.v_par[:, :, nan, 0] = float("nan")
    q = torch.ones(1, N, G * Hkv, dh, dtype=dtype, device=DEV)
    length = torch.tensor([L], dtype=torch.int32, device=DEV)
    return api.medusa_tree_attention_packed(q, c, length, api.Tree(*tree), 0.1)


@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("nan,big", [(5, 690), (690, 5), (5, 150), (150, 5), (5, 21)])
@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_nan_row_of_weight_zero_is_kept(kernel, chunks, nan, big, which):
    if chunks == "many" and 690 in (nan, big):
        nan, big = (nan, 7890) if big == 690 else (7890, big)
    out = _call(kernel, chunks, nan, big, which)
    assert bool(out.isnan().all())
    assert api.device_status() == 0


@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("kernel", KERNELS)
def test_without_it_the_large_key_answers(kernel, chunks):
    """The same inputs without the NaN: the value of the large key, which has all
    the weight."""
    tree, G, dh, dtype = KERNELS[kernel]
    out = _call(kernel, chunks, 0, 300, "")
    assert bool(out.isfinite().all()) and out.abs().max() <= 0.05 * 8 * (1 + 2.0 ** -7)
    assert api.device_status() == 0
