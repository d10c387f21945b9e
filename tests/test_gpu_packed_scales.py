"""GPU: tree attention over the 4-bit cache at the edges of the row scales:
zero, not a number, tiny, each through every kernel."""
import math

import pytest
import torch

import ext_reference as R
from oracle import medusa_oracle as O
from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

# (tree (K, s, N), query heads per kv-head, dh, dtype, rounding of the kernel that takes it)
KERNELS = {
    "rows8": ((4, 3, 5), 1, 128, BF, "fp16"),
    "rows16": ((4, 3, 5), 3, 128, BF, "fp16"),
    "keys32": ((4, 3, 9), 3, 128, BF, "fp16"),
    "keys64": ((5, 10, 50), 1, 128, BF, "fp16"),
    "keys128": ((5, 10, 50), 2, 128, BF, "fp16"),
    "pair": ((5, 3, 200), 1, 128, BF, "fp16v"),
    "simt64": ((4, 3, 30), 2, 64, BF, "fp32"),
    "simt_f32": ((5, 3, 40), 1, 128, F32, "fp32"),
}


def _inputs(kernel, Ls, Hkv=2, scale_q=1.0):
    (tree, G, dh, dtype, _), N = KERNELS[kernel], KERNELS[kernel][0][2]
    g = torch.Generator(device=DEV).manual_seed(len(Ls) * 131 + N + G)
    B, Lcap = len(Ls), (max(Ls) + N + 8) // 4 * 4
    q = (torch.randn(B, N, G * Hkv, dh, generator=g, device=DEV) * scale_q).to(dtype)
    c = api.PackedCache.empty(B, Hkv, Lcap, dh, DEV)
    for x in (c.k_codes, c.v_codes):
        x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV, dtype=torch.int16))
    for p in (c.k_par, c.v_par):
        p[..., 0] = torch.rand(p.shape[:-1], generator=g, device=DEV).mul_(3).exp2_().mul_(0.08)
        p[..., 1] = torch.randint(4, 12, p.shape[:-1], generator=g, device=DEV).float()
    return q, c, torch.tensor(Ls, dtype=torch.int32, device=DEV), tree


def _check(kernel, q, c, L, tree, scale, rows=None, window=0, sinks=0):
    """The call against the 64-bit form, at the output rows where `rows` holds."""
    got = api.medusa_tree_attention_packed(q, c, L, api.Tree(*tree), scale, window, sinks)
    ref = R.attention(q, R.decode(c.k_codes, c.k_par), R.decode(c.v_codes, c.v_par), L.tolist(),
                      O.tree_plan(*tree), scale, window, sinks)
    if rows is not None:
        ref = [x[rows] for x in ref]
    R.assert_close(got if rows is None else got[rows], *ref, q.dtype, KERNELS[kernel][4], kernel)
    assert api.device_status() == 0
    return got


@pytest.mark.parametrize("scale_q", [1e-3, 1.0])
@pytest.mark.parametrize("part", ["all", "tree", "first", "last"])
@pytest.mark.parametrize("kernel", KERNELS)
def test_key_tiles_of_zeros(kernel, part, scale_q):
    """K rows of zeros (scale 0): every key, the tree's tile (the prefix ends
    with a tile), the first tile, the last tile in use."""
    q, c, L, tree = _inputs(kernel, [256, 300], scale_q=scale_q)
    lo, hi = {"all": (0, None), "tree": (256, None), "first": (0, 128), "last": (384, None)}[part]
    c.k_par[:, :, lo:hi] = 0
    c.k_codes[:, :, lo:hi] = 0
    scale = 1 / math.sqrt(q.shape[-1])
    for w, s in ((0, 0), (140, 3)):
        _check(kernel, q, c, L, tree, scale, window=w, sinks=s)


@pytest.mark.parametrize("scale,scale_q", [(0.088, 1e-3), (1e-6, 1.0), (0.088, 1.0)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_cache_of_zeros(kernel, scale, scale_q):
    q, c, L, tree = _inputs(kernel, [0, 130], scale_q=scale_q)
    c = api.PackedCache.empty(2, c.Hkv, c.Lcap, c.dh, DEV)
    out = api.medusa_tree_attention_packed(q, c, L, api.Tree(*tree), scale)
    assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_nan_row_in_a_tile_of_zeros(kernel):
    """The tree's tile holds K rows of zeros and one with scale NaN: exactly the
    nodes that see that one are NaN, the others follow the formula."""
    q, c, L, tree = _inputs(kernel, [256, 128], scale_q=1e-3)
    c.k_par[0, :, 256:] = 0
    c.k_par[1, :, 128:] = 0
    for b, Lb in enumerate(L.tolist()):
        c.k_par[b, :, Lb + 2] = math.nan
    depth, anc = R.tree_masks(O.tree_plan(*tree))
    sees = anc[:, 2].to(DEV)
    rows = (~sees)[None, :, None].expand(q.shape[:3])
    got = _check(kernel, q, c, L, tree, 0.088, rows=rows)
    assert bool(got[:, sees].isnan().all())


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("exp", [110, 116, 117, 118])
@pytest.mark.parametrize("kernel", KERNELS)
def test_tiny_scales(kernel, exp, which):
    """Rows whose scales are all 2^-exp, some K rows zeros; codes of V on one
    side of zero, so that the outputs stay normal numbers of their type."""
    q, c, L, tree = _inputs(kernel, [256, 300])
    if which != "v":
        c.k_par[..., 0] = 2.0 ** -exp
        c.k_par[:, :, ::7] = 0
    if which != "k":
        c.v_par[..., 0] = 2.0 ** -exp
        c.v_par[..., 1] = 0
        c.v_codes.bitwise_or_(0x88)
    _check(kernel, q, c, L, tree, 0.088)


@pytest.mark.parametrize("kernel", KERNELS)
def test_value_scales_that_start_tiny(kernel):
    """Scales of 2^-118 in the first tiles, ordinary ones after them."""
    q, c, L, tree = _inputs(kernel, [600, 300])
    c.v_par[:, :, :200, 0] = 2.0 ** -118
    c.k_par[:, :, :200, 0] = 2.0 ** -118
    _check(kernel, q, c, L, tree, 0.088)
