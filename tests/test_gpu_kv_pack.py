"""GPU: storing rows in the 4-bit cache, reading them back and compacting the
accepted path, bit for bit against the definition."""
import math

import pytest
import torch

import ext_reference as R
from medusa_head_speculative_02_b200 import _lib as lib
from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rows(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _poisoned(B, H, Lcap, dh, layers=None):
    c = api.PackedCache.empty(B, H, Lcap, dh, DEV, layers)
    c.k_codes.fill_(0xA5)
    c.v_codes.fill_(0x5A)
    c.k_par.fill_(7.5)
    c.v_par.fill_(-3.25)
    return c


def _expect(cache, k, v, start, count):
    """The cache's arrays after the store, on the CPU."""
    arrs = [t.clone().cpu() for t in (cache.k_codes, cache.k_par, cache.v_codes, cache.v_par)]
    B, T = k.shape[:2]
    for x, ci in ((k, 0), (v, 2)):
        codes, scale, zero = R.encode(x)
        for b in range(B):
            for t in range(min(T, count[b])):
                slot = start[b] + t
                if 0 <= slot < cache.Lcap:
                    arrs[ci][b, :, slot] = codes[b, t]
                    arrs[ci + 1][b, :, slot, 0] = scale[b, t].to(torch.bfloat16)
                    arrs[ci + 1][b, :, slot, 1] = zero[b, t].to(torch.bfloat16)
    return arrs


def _same(a, b):
    if a.dtype == torch.bfloat16:
        return bool(((a == b) | (a.isnan() & b.isnan())).all())
    return torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,H,dh,Lcap,start,count", [
    (1, 1, 1, 128, 4, [0], None),
    (1, 64, 32, 128, 132, [65], None),
    (3, 17, 5, 64, 40, [0, 23, 30], [17, 1, 9]),
    (2, 9, 7, 128, 12, [-3, 8], [9, 9]),            # slots below 0 and past the end
    (4, 33, 3, 128, 64, [31, 0, 5, 2], [0, -4, 40, 33]),  # empty, negative and large counts
    (2, 700, 8, 128, 1024, [100, 324], [700, 655]),  # four rows per lane group
])
def test_pack_matches_the_definition(dtype, B, T, H, dh, Lcap, start, count):
    k, v = _rows((B, T, H, dh), dtype, 1), _rows((B, T, H, dh), dtype, 2) * 3 + 1
    v = v.to(dtype)
    cache = _poisoned(B, H, Lcap, dh)
    want = _expect(cache, k, v, start, count or [T] * B)
    st = torch.tensor(start, dtype=torch.int32, device=DEV)
    ct = None if count is None else torch.tensor(count, dtype=torch.int32, device=DEV)
    api.medusa_kv_pack(k.to(DEV), v.to(DEV), cache, st, ct)
    got = [t.cpu() for t in (cache.k_codes, cache.k_par, cache.v_codes, cache.v_par)]
    for g, w in zip(got, want):
        assert _same(g, w)
    # reading back: the values the rows stand for, zeros elsewhere
    for odt in (torch.float32, torch.bfloat16):
        outs = api.medusa_kv_unpack(cache, st, T, odt, ct)
        for o, codes, par in ((outs[0], want[0], want[1]), (outs[1], want[2], want[3])):
            ref = torch.zeros(B, T, H, dh, dtype=torch.float64)
            vals = R.decode(codes, par)
            for b in range(B):
                for t in range(T):
                    slot = start[b] + t
                    if (count is None or t < count[b]) and 0 <= slot < Lcap:
                        ref[b, t] = vals[b, :, slot]
            assert torch.equal(o.cpu(), ref.to(odt))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_the_edges_of_the_types(dtype):
    dh = 128
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    rows = [torch.zeros(dh), torch.full((dh,), 2.5), torch.full((dh,), -0.75),
            torch.linspace(0, 15, dh), torch.linspace(-15, 0, dh),
            torch.arange(dh).float() % 31 / 2 - 7.5,          # ties at every half
            torch.full((dh,), math.nan), torch.linspace(-1, 1, dh), torch.linspace(-1, 1, dh),
            torch.linspace(-1, 1, dh) * big, torch.linspace(0, 1, dh) * big,
            torch.linspace(-1, 1, dh) * tiny, torch.linspace(-1, 1, dh) * tiny * 64,
            torch.linspace(-1, 1, dh) * 1e-30, torch.full((dh,), -0.0)]
    rows[7][5] = math.inf
    rows[8][127] = math.nan
    x = torch.stack(rows).to(dtype)[None, :, None, :].contiguous()
    T = x.shape[1]
    cache = _poisoned(1, 1, 16, dh)
    want = _expect(cache, x, x.flip(-1), [0], [T])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.medusa_kv_pack(x.to(DEV), x.flip(-1).contiguous().to(DEV), cache, st)
    got = [t.cpu() for t in (cache.k_codes, cache.k_par, cache.v_codes, cache.v_par)]
    for g, w in zip(got, want):
        assert _same(g, w)
    k, _ = api.medusa_kv_unpack(cache, st, T, torch.float32)
    k = k.cpu()[0, :, 0]
    assert k[0].abs().max() == 0 and k[14].abs().max() == 0
    for i in (6, 7, 8):
        assert k[i].isnan().all()
    # a finite row is off by at most half a step, and by bf16's rounding of the
    # scale (15 codes of it) where the row's end is clamped
    for i in (1, 2, 3, 4, 5):
        xi = x[0, i, 0].double()
        s = float(want[1][0, 0, i, 0])
        assert (k[i].double() - xi).abs().max() <= s * (0.5 + 15 * 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.float32])
def test_pack_near_ties(dtype):
    """Quotients within a few ulp of a tie are decided by the correctly
    rounded fp32 quotient."""
    dh, n = 128, 64
    g = torch.Generator().manual_seed(5)
    x = torch.empty(1, n, 1, dh)
    for i in range(n):
        s = float((torch.rand((), generator=g) + 0.5).bfloat16())
        q = torch.randint(-7, 8, (dh,), generator=g).float() + 0.5
        u = (torch.randint(-3, 4, (dh,), generator=g).float() * 2.0 ** -22)
        x[0, i, 0] = (q * s) * (1 + u)
        x[0, i, 0, 0], x[0, i, 0, 1] = -7.5 * s, 7.5 * s   # pins the scale
    cache = _poisoned(1, 1, n, dh)
    want = _expect(cache, x, x, [0], [n])
    api.medusa_kv_pack(x.to(DEV), x.to(DEV), cache, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.equal(cache.k_codes.cpu(), want[0])


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("dh", [64, 128])
def test_compact_moves_rows_bit_for_bit(layers, dh):
    B, H, Lcap, K = 6, 5, 40, 4
    c = _poisoned(B, H, Lcap, dh, layers)
    g = torch.Generator().manual_seed(3)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_par, c.v_par):
        t.copy_(torch.randn(t.shape, generator=g))
    L = [3, 0, 20, 7, 30, -1]
    alen = [4, 0, 2, 5, 3, 2]                     # 5: outside [0, K]
    nodes = [[0, 1, 4, 9, 12], [0, -1, -1, -1, -1], [0, 3, 3, -1, -1], [0, 1, 2, 3, 4],
             [0, 2, 1, 11, -1], [0, 1, 2, -1, -1]]  # a node below its step, a slot past the end
    arrs = [t.clone().cpu() for t in (c.k_codes, c.k_par, c.v_codes, c.v_par)]
    for t in arrs:
        for b in range(B):
            if L[b] < 0 or not 0 <= alen[b] <= K:
                continue
            for j in range(1, alen[b] + 1):
                n = nodes[b][j]
                if n >= j and L[b] + n < Lcap:
                    t[..., b, :, L[b] + j, :] = t[..., b, :, L[b] + n, :]
    i32 = dict(dtype=torch.int32, device=DEV)
    new = api.medusa_kv_compact_packed(c, torch.tensor(L, **i32), torch.tensor(alen, **i32),
                                       torch.tensor(nodes, **i32), K)
    for t, w in zip((c.k_codes, c.k_par, c.v_codes, c.v_par), arrs):
        assert torch.equal(t.cpu(), w)
    assert new.cpu().tolist() == [8, 1, 23, -1, 34, -1]
    # the index-checked library records the bad entries (and this clears them)
    assert api.device_status() == (lib.ERR_BOUNDS if lib.DEBUG else 0)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes of codes: the last sequence's rows land
    in its own slots."""
    B, H, Lcap, dh = 5, 32, 524288, 128   # 5.4 GB per code array
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB free")
    c = api.PackedCache.empty(B, H, Lcap, dh, DEV)
    k, v = _rows((B, 3, H, dh), torch.bfloat16, 8).to(DEV), _rows((B, 3, H, dh), torch.bfloat16, 9).to(DEV)
    st = torch.full((B,), Lcap - 3, dtype=torch.int32, device=DEV)
    api.medusa_kv_pack(k, v, c, st)
    codes, _, _ = R.encode(v)
    assert torch.equal(c.v_codes[:, :, -3:].cpu(), codes.transpose(1, 2))
    assert int(c.v_codes[:, :, :-3].max()) == 0
    kk, vv = api.medusa_kv_unpack(c, st, 3, torch.float32)
    ref = R.decode(c.v_codes[4, :, -3:], c.v_par[4, :, -3:]).float().transpose(0, 1)
    assert torch.equal(vv[4], ref)
    q = torch.randn(B, 1, H, dh, device=DEV).bfloat16()
    L = torch.full((B,), Lcap - 1, dtype=torch.int32, device=DEV)
    # the window holds only the last three slots, whose values are known
    out = api.medusa_tree_attention_packed(q, c, L, api.Tree(1, 1, 1), 1 / math.sqrt(dh), window=3)
    kd, vd = (R.decode(x[:, :, -3:], p[:, :, -3:]) for x, p in ((c.k_codes, c.k_par), (c.v_codes, c.v_par)))
    p = torch.softmax(torch.einsum("bhd,bhkd->bhk", q[:, 0].double(), kd) / math.sqrt(dh), -1)
    ref = torch.einsum("bhk,bhkd->bhd", p, vd)
    assert (out[:, 0].double() - ref).abs().max() <= 2.0 ** -8 * vd.abs().max()


def test_empty_calls_and_a_captured_store():
    B, H, dh = 2, 3, 128
    c = _poisoned(B, H, 32, dh)
    before = c.k_codes.clone()
    st = torch.zeros(B, dtype=torch.int32, device=DEV)
    api.medusa_kv_pack(torch.empty(B, 0, H, dh, device=DEV), torch.empty(B, 0, H, dh, device=DEV), c, st)
    assert torch.equal(c.k_codes, before)
    k, v = (_rows((B, 5, H, dh), torch.bfloat16, s).to(DEV) for s in (1, 2))
    api.medusa_kv_pack(k, v, c, st)   # library set-up outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.medusa_kv_pack(k, v, c, st)
        outs = api.medusa_kv_unpack(c, st, 5, torch.float32)
    k.copy_(_rows((B, 5, H, dh), torch.bfloat16, 11))
    st.fill_(9)
    g.replay()
    torch.cuda.synchronize()
    codes, scale, zero = R.encode(k)
    assert torch.equal(c.k_codes[:, :, 9:14].cpu(), codes.transpose(1, 2))
    par = torch.stack([scale, zero], -1).to(torch.bfloat16)
    assert torch.equal(outs[0].cpu(), R.decode(codes, par).float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("exp", [0, -60, 100, -97])
def test_quotients_at_and_beside_ties(dtype, exp):
    """Values at (n + 1/2) scale, as far as the type holds them, and their
    neighbours, for every significand of hi and several shares of lo: codes as
    the definition's rounding to even gives them."""
    g = torch.Generator().manual_seed(7)
    hi = (128 + torch.arange(128, dtype=torch.float64)) * 2.0 ** (exp - 7)
    rows = []
    for share in (0.0, 0.3, 1.0, 2.5):
        lo = -(hi * share).to(torch.bfloat16).double()
        scale = ((hi - lo).float() / 15).to(torch.bfloat16).double()
        n = torch.arange(-16, 16, dtype=torch.float64)
        tie = ((n + 0.5) * scale[:, None]).to(dtype)
        up = torch.nextafter(tie, torch.full_like(tie, math.inf))
        down = torch.nextafter(tie, torch.full_like(tie, -math.inf))
        rnd = (torch.rand(128, 30, generator=g, dtype=torch.float64) * (hi - lo)[:, None] + lo[:, None])
        x = torch.cat([tie, up, down, rnd.to(dtype)], 1).double()
        x = torch.minimum(torch.maximum(x, lo[:, None]), hi[:, None])
        rows.append(torch.cat([x, lo[:, None], hi[:, None]], 1).to(dtype))
    x = torch.stack(rows).view(4, 128, 1, 128).contiguous()
    cache = _poisoned(4, 1, 128, 128)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    want = _expect(cache, x, -x, [0] * 4, [128] * 4)
    api.medusa_kv_pack(x.to(DEV), (-x).to(DEV), cache, st)
    for a, w in zip((cache.k_codes, cache.k_par, cache.v_codes, cache.v_par), want):
        assert _same(a.cpu(), w)
