"""Measured cases of the operators on a 4-bit KV cache and on a sliding window.

Four passes, each in a plain form (elementary torch operations) and as calls
of the framework:

  pack     K/V rows of new tokens written to the 4-bit cache, and the written
           slots read back as values (prefill, ragged batches, one tree)
  packed   tree attention over the 4-bit cache, full or windowed
  window   tree attention over the bf16/fp32 cache, sliding window with sinks
  keep     the tail of a verify step on the 4-bit cache: the tree's K/V are
           stored, the accepted path is compacted, its slots are read back

Row format of the 4-bit cache, per (sequence, kv-head, slot) row x of dh
values: lo = min(0, min x), hi = max(0, max x), scale = bf16((hi - lo) / 15),
zero = clamp(rint(-lo / scale), 0, 15), code = clamp(rint(x / scale) + zero,
0, 15), and the row stands for scale * (code - zero).  Element 2i is the low
half of byte i.  Codes are [B][Hkv][Lcap][dh / 2] bytes, (scale, zero) pairs
[B][Hkv][Lcap][2] bf16.  rint rounds ties to even.

Visible keys of tree node i at depth D of a sequence with prefix length L,
window W and S sinks (W = 0: no window): prefix slots and the slots L + a of
the node's ancestors a and of itself, each at position p (a prefix slot its
index, a node L + its depth), restricted to p < S or p > L + D - W.
"""
import heapq
import math
from fractions import Fraction

import torch

own = False

_BF, _F32 = "bf16", "f32"
_DT = {_BF: torch.bfloat16, _F32: torch.float32}

# The costliest listed cases bound what a drawn case may cost.
_MAX_FLOPS = 9.0e11
_MAX_VALUES = 8.8e8


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one verify step's tree stored for a 7B-shaped layer: latency only
        dict(name="pack_tree_7b", op="pack", dt=_BF, B=1, T=64, Hkv=32, dh=128, ragged=0),
        # ragged prefill of a GQA model: 16 prompts of 700 to 8192 tokens
        dict(name="pack_prefill_gqa", op="pack", dt=_BF, B=16, T=8192, Hkv=8, dh=128, ragged=1),
        # 7B-shaped verify step, one sequence: few keys, every SM wanted
        dict(name="packed_7b_b1", op="packed", dt=_BF, B=1, K=5, s=10, N=64, Hq=32, Hkv=32, dh=128,
             L_lo=2048, L_hi=2048, window=0, sinks=0),
        # 8B-GQA-shaped verify step: 512 query rows per kv-head
        dict(name="packed_8b_gqa_b16", op="packed", dt=_BF, B=16, K=5, s=8, N=128, Hq=32, Hkv=8,
             dh=128, L_lo=8192, L_hi=8192, window=0, sinks=0),
        # plain decoding of a ragged GQA batch over long prefixes: single tokens
        dict(name="packed_token_long", op="packed", dt=_BF, B=16, K=1, s=1, N=1, Hq=32, Hkv=8, dh=128,
             L_lo=9001, L_hi=32768, window=0, sinks=0),
        # the long-context verify step: 256-node trees over 32K prefixes
        dict(name="packed_longctx_b4", op="packed", dt=_BF, B=4, K=5, s=3, N=256, Hq=52, Hkv=52,
             dh=128, L_lo=32768, L_hi=32768, window=0, sinks=0),
        # the fp32 path at the smallest configuration
        dict(name="packed_tiny_f32", op="packed", dt=_F32, B=1, K=4, s=3, N=16, Hq=4, Hkv=4, dh=64,
             L_lo=128, L_hi=128, window=0, sinks=0),
        # 7B-shaped step with a short window: latency of a few tiles
        dict(name="window_7b_b1", op="window", dt=_BF, B=1, K=5, s=10, N=64, Hq=32, Hkv=32, dh=128,
             L_lo=2048, L_hi=2048, window=512, sinks=4),
        # the long-context step's heads and tree, windowed
        dict(name="window_longctx_b4", op="window", dt=_BF, B=4, K=5, s=3, N=256, Hq=52, Hkv=52,
             dh=128, L_lo=32768, L_hi=32768, window=4096, sinks=16),
        # single tokens of a ragged GQA batch, window of an odd size
        dict(name="window_token", op="window", dt=_BF, B=16, K=1, s=1, N=1, Hq=32, Hkv=8, dh=128,
             L_lo=1, L_hi=8192, window=4095, sinks=4),
        # tail of a verify step, ragged 13B-shaped batch
        dict(name="keep_13b_b8", op="keep", dt=_BF, B=8, K=5, s=10, N=64, Hkv=40, dh=128,
             L_lo=1024, L_hi=4096),
        # the same at the 8B-GQA shape
        dict(name="keep_8b_gqa_b16", op="keep", dt=_BF, B=16, K=5, s=8, N=128, Hkv=8, dh=128,
             L_lo=8192, L_hi=8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _tree_size(rng):
    K, s = rng.choice([(1, 1), (2, 4), (4, 3), (5, 3), (5, 8), (5, 10), (8, 2)])
    room = sum(s ** d for d in range(K + 1))
    return K, s, min(room, _log_int(rng, 1, 256))


def draw(rng):
    op = rng.choice(["pack", "packed", "packed", "window", "window", "keep"])
    dt = _BF if rng.random() < 0.85 else _F32
    dh = 128 if rng.random() < 0.8 else 64
    if op == "pack":
        B, Hkv = _log_int(rng, 1, 16), rng.choice([1, 2, 4, 5, 8, 32, 40])
        T = min(_log_int(rng, 1, 8192), max(1, int(_MAX_VALUES / 7 / (B * Hkv * dh))))
        return dict(op=op, dt=dt, B=B, T=T, Hkv=Hkv, dh=dh, ragged=rng.randrange(2))
    if op == "keep":
        K, s, N = _tree_size(rng)
        hi = _log_int(rng, 8, 8192)
        return dict(op=op, dt=dt, B=_log_int(rng, 1, 16), K=K, s=s, N=N, Hkv=rng.choice([1, 5, 8, 40]),
                    dh=dh, L_lo=rng.randint(0, hi), L_hi=hi)
    K, s, N = _tree_size(rng)
    Hkv = rng.choice([1, 2, 4, 5, 8, 32, 40, 52])
    G = rng.choice([1, 1, 2, 4, 7, 8]) if Hkv <= 8 else 1
    B = _log_int(rng, 1, 16)
    hi = _log_int(rng, 1, 32768)
    windowed = op == "window" or rng.random() < 0.35
    es = 2 if dt == _BF else 4
    fl = 4.0 * B * N * Hkv * G * dh
    if dt == _F32 or dh == 64:
        fl *= 8  # the ranges of these paths are those of the small configurations
    hi = max(1, min(hi, int(_MAX_FLOPS / fl), int(_MAX_VALUES / es * 2 / (B * Hkv * dh))))
    return dict(op=op, dt=dt, B=B, K=K, s=s, N=N, Hq=Hkv * G, Hkv=Hkv, dh=dh,
                L_lo=rng.randint(max(0, hi // 4), hi), L_hi=hi,
                window=_log_int(rng, 1, 8192) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 16, 130]) if windowed else 0)


# -------------------------------------------------------------------- inputs
def _lcap(case):
    """Slots of the cache: the longest prefix, the tree, rounded up to 4."""
    return (case["L_hi"] + case["N"] + 3) // 4 * 4


def _tree_plan(K, s, N):
    """Depth of every node and the ancestor-or-self matrix: the N rank tuples
    of largest 0.8^depth * 0.5^(sum of ranks), ties by depth then order."""
    heap, kept = [(Fraction(-1), 0, ())], []
    while len(kept) < N:
        neg, d, r = heapq.heappop(heap)
        kept.append((d, r))
        if d < K:
            heapq.heappush(heap, (neg * Fraction(4, 5), d + 1, r + (0,)))
        if r and r[-1] + 1 < s:
            heapq.heappush(heap, (neg / 2, d, r[:-1] + (r[-1] + 1,)))
    kept.sort()
    index = {r: i for i, (_, r) in enumerate(kept)}
    anc = torch.zeros(N, N, dtype=torch.bool)
    for i, (d, r) in enumerate(kept):
        for e in range(d + 1):
            anc[i, index[r[:e]]] = True
    return torch.tensor([d for d, _ in kept], dtype=torch.int64), anc


def _gen(seed, tid):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + tid * 7919 + 17)
    return g


def _randn(shape, dtype, seed, tid):
    return torch.randn(shape, generator=_gen(seed, tid), device="cuda").to(dtype)


def _kv_rows(shape, dtype, seed, tid):
    """K or V rows [..., dh]: N(0, 1) with a fixed per-channel offset, as
    projections with a few strong channels give."""
    x = torch.randn(shape, generator=_gen(seed, tid), device="cuda")
    off = torch.randn(shape[-2:], generator=_gen(seed, tid + 50), device="cuda")
    return x.add_(off, alpha=0.5).to(dtype)


def _ints(lo, hi, n, seed, tid):
    return torch.randint(lo, hi + 1, (n,), generator=_gen(seed, tid), device="cuda",
                         dtype=torch.int64).to(torch.int32)


def _random_cache(B, H, Lcap, dh, seed, tid):
    """Codes and (scale, zero) of a filled cache, made in slices of heads."""
    codes = torch.empty(B, H, Lcap, dh // 2, dtype=torch.uint8, device="cuda")
    par = torch.empty(B, H, Lcap, 2, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        x = _kv_rows((Lcap, H, dh), torch.bfloat16, seed, tid + 100 * (b + 1))
        codes[b], par[b] = _encode(x.transpose(0, 1))
        del x
    return codes, par


def prepare(case, seed):
    dt, B, dh = _DT[case["dt"]], case["B"], case["dh"]
    st = dict(case=case)
    op = case["op"]
    if op == "pack":
        T, H = case["T"], case["Hkv"]
        st["k"] = _kv_rows((B, T, H, dh), dt, seed, 1)
        st["v"] = _kv_rows((B, T, H, dh), dt, seed, 2)
        lo = max(1, T // 12) if case["ragged"] else T
        st["count"] = _ints(lo, T, B, seed, 3)
        st["start"] = _ints(0, 64, B, seed, 4)
        lcap = (T + 64 + 3) // 4 * 4
        st["cache"] = [torch.zeros(B, H, lcap, dh // 2, dtype=torch.uint8, device="cuda"),
                       torch.zeros(B, H, lcap, 2, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(B, H, lcap, dh // 2, dtype=torch.uint8, device="cuda"),
                       torch.zeros(B, H, lcap, 2, dtype=torch.bfloat16, device="cuda")]
        _own_state(st)
        return st
    N, H, lcap = case["N"], case["Hkv"], _lcap(case)
    depth, anc = _tree_plan(case["K"], case["s"], N)
    st["depth"], st["anc"] = depth.cuda(), anc.cuda()
    st["L"] = _ints(case["L_lo"], case["L_hi"], B, seed, 5)
    if op == "keep":
        st["k"] = _kv_rows((B, N, H, dh), dt, seed, 1)
        st["v"] = _kv_rows((B, N, H, dh), dt, seed, 2)
        # an accepted path: from the root to a node drawn per sequence
        pick = _ints(0, N - 1, B, seed, 6).cpu().tolist()
        nodes = torch.full((B, case["K"] + 1), -1, dtype=torch.int32)
        for b, n in enumerate(pick):
            path = torch.nonzero(anc[n]).flatten().to(torch.int32)
            nodes[b, :path.numel()] = path
        st["nodes"] = nodes.cuda()
        st["alen"] = depth[pick].to(torch.int32).cuda()
        st["cache"] = [*_random_cache(B, H, lcap, dh, seed, 10),
                       *_random_cache(B, H, lcap, dh, seed, 20)]
        _own_state(st)
        return st
    st["q"] = _randn((B, N, case["Hq"], dh), dt, seed, 7)
    if op == "packed":
        st["cache"] = [*_random_cache(B, H, lcap, dh, seed, 10),
                       *_random_cache(B, H, lcap, dh, seed, 20)]
    else:
        st["k"] = _randn((B, lcap, H, dh), dt, seed, 8)
        st["v"] = _randn((B, lcap, H, dh), dt, seed, 9)
    _own_state(st)
    return st


def _own_state(st):
    """What a program of this framework keeps between calls: the tree plan,
    the cache object, output and scratch buffers."""
    if not own or "api" in st:
        return
    from medusa_head_speculative_02_b200 import api
    c = st["case"]
    st["api"] = api
    if "cache" in st:
        st["packed"] = api.PackedCache(*st["cache"])
    if c["op"] in ("packed", "window"):
        t = st["tree"] = api.Tree(c["K"], c["s"], c["N"])
        st["out"] = torch.empty_like(st["q"])
        size = api.attention_packed_workspace_size if c["op"] == "packed" \
            else api.attention_window_workspace_size
        n = size(t, c["B"], c["Hq"], c["Hkv"], c["dh"], _lcap(c), st["q"].dtype, c["window"],
                 c["sinks"])
        st["ws"] = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------- plain form
def _encode(x):
    """Rows x [..., dh] -> (codes uint8 [..., dh / 2], (scale, zero) bf16 [..., 2])."""
    x = x.float()
    lo = x.amin(-1, keepdim=True).clamp(max=0.0)
    hi = x.amax(-1, keepdim=True).clamp(min=0.0)
    scale = ((hi - lo) / 15.0).to(torch.bfloat16)
    div = torch.where(scale > 0, scale, torch.ones_like(scale)).float()
    zero = torch.round(-lo / div).clamp(0.0, 15.0)
    c = torch.round(x / div).add_(zero).clamp_(0.0, 15.0).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([scale, zero.to(torch.bfloat16)], -1)


def _decode(codes, par):
    """The fp32 values that rows of codes stand for."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    p = par.float()
    return (c - p[..., 1:2]).mul_(p[..., 0:1])


def _store(cache, k, v, start, count):
    B, T = k.shape[:2]
    t = torch.arange(T, device=k.device)
    live = t[None] < count[:, None]
    b, tt = torch.nonzero(live, as_tuple=True)
    slot = start.long()[b] + tt
    for x, codes, par in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        c, p = _encode(x[b, tt])
        codes[b, :, slot] = c
        par[b, :, slot] = p


def _read(cache, start, count, T, dtype):
    B, H, Lcap, half = cache[0].shape
    t = torch.arange(T, device=start.device)
    live = t[None] < count[:, None]
    b, tt = torch.nonzero(live, as_tuple=True)
    slot = start.long()[b] + tt
    outs = []
    for codes, par in ((cache[0], cache[1]), (cache[2], cache[3])):
        out = torch.zeros(B, T, H, 2 * half, dtype=dtype, device=codes.device)
        out[b, tt] = _decode(codes[b, :, slot], par[b, :, slot]).to(dtype)
        outs.append(out)
    return outs


def _visible(depth, anc, L, window, sinks, n_keys):
    """Truth values [N][n_keys]: which slots each node sees."""
    N = depth.numel()
    slot = torch.arange(n_keys, device=depth.device)
    tree = slot >= L
    node = (slot - L).clamp(0, N - 1)
    pos = torch.where(tree, L + depth[node], slot)
    vis = torch.where(tree[None], anc[:, node], torch.ones_like(anc[:, node]))
    if window > 0:
        vis = vis & ((pos[None] < sinks) | (pos[None] > L + depth[:, None] - window))
    return vis


def _attend(q, k, v, vis, scale):
    """q [N][H][G][dh], k and v [H][keys][dh] in fp32, vis [N][keys]."""
    s = torch.matmul(q.permute(1, 2, 0, 3), k[:, None].transpose(-1, -2))
    s = s.mul_(scale).masked_fill_(~vis, float("-inf"))
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(s, v[:, None]) / s.sum(-1, keepdim=True)
    return out.permute(2, 0, 1, 3)


def _plain_attention(st):
    c, q = st["case"], st["q"]
    B, N, Hq, dh = q.shape
    H = c["Hkv"]
    out = torch.empty_like(q)
    scale = 1.0 / math.sqrt(dh)
    for b, L in enumerate(st["L"].tolist()):
        vis = _visible(st["depth"], st["anc"], L, c["window"], c["sinks"], L + N)
        idx = torch.nonzero(vis.any(0)).flatten()
        full = idx.numel() == L + N
        step = max(1, int(3e8 / (idx.numel() * N * (Hq // H))))
        for h in range(0, H, step):
            hs = slice(h, h + step)
            if c["op"] == "packed":
                parts = [x[b, hs, :L + N] if full else x[b, hs][:, idx] for x in st["cache"]]
                k, v = _decode(*parts[:2]), _decode(*parts[2:])
            else:
                k, v = ((x[b, :L + N, hs] if full else x[b, idx][:, hs]).transpose(0, 1).float()
                        for x in (st["k"], st["v"]))
            qh = q[b].float().view(N, H, Hq // H, dh)[:, hs]
            o = _attend(qh, k, v, vis if full else vis[:, idx], scale)
            out[b].view(N, H, Hq // H, dh)[:, hs] = o.to(q.dtype)
    return out


def _plain(st):
    c = st["case"]
    if c["op"] == "pack":
        _store(st["cache"], st["k"], st["v"], st["start"], st["count"])
        return _read(st["cache"], st["start"], st["count"], c["T"], _DT[c["dt"]])
    if c["op"] == "keep":
        B, N, K = c["B"], c["N"], c["K"]
        every = torch.full_like(st["L"], N)
        _store(st["cache"], st["k"], st["v"], st["L"], every)
        j = torch.arange(1, K + 1, device="cuda")
        b, jj = torch.nonzero(j[None] <= st["alen"][:, None], as_tuple=True)
        src = st["L"].long()[b] + st["nodes"][b, jj + 1]
        for x in st["cache"]:
            x[b, :, st["L"].long()[b] + jj + 1] = x[b, :, src]
        new_len = st["L"] + 1 + st["alen"]
        return [new_len, *_read(st["cache"], st["L"], st["alen"] + 1, K + 1, _DT[c["dt"]])]
    return _plain_attention(st)


# ---------------------------------------------------------------------- passes
def run(state):
    if not own:
        return _plain(state)
    _own_state(state)
    api, c = state["api"], state["case"]
    if c["op"] == "pack":
        api.medusa_kv_pack(state["k"], state["v"], state["packed"], state["start"], state["count"])
        return api.medusa_kv_unpack(state["packed"], state["start"], c["T"], _DT[c["dt"]],
                                    state["count"])
    if c["op"] == "keep":
        api.medusa_kv_pack(state["k"], state["v"], state["packed"], state["L"])
        new_len = api.medusa_kv_compact_packed(state["packed"], state["L"], state["alen"],
                                               state["nodes"], c["K"])
        return [new_len, *api.medusa_kv_unpack(state["packed"], state["L"], c["K"] + 1,
                                               _DT[c["dt"]], state["alen"] + 1)]
    scale = 1.0 / math.sqrt(c["dh"])
    if c["op"] == "packed":
        return api.medusa_tree_attention_packed(state["q"], state["packed"], state["L"],
                                                state["tree"], scale, window=c["window"],
                                                sinks=c["sinks"], out=state["out"], ws=state["ws"])
    return api.medusa_tree_attention_window(state["q"], state["k"], state["v"], state["L"],
                                            state["tree"], scale, c["window"], c["sinks"],
                                            out=state["out"], ws=state["ws"])


def work(case):
    B, dh = case["B"], case["dh"]
    es = 2 if case["dt"] == _BF else 4
    row = dh // 2 + 4
    op = case["op"]
    if op == "pack":
        T, H = case["T"], case["Hkv"]
        lo = max(1, T // 12) if case["ragged"] else T
        live = B * (lo + T) / 2 * H * 2            # K and V rows expected
        return {"bytes": live * (dh * es + row) + 2 * B * T * H * dh * es, "flops": live * dh * 4}
    N, H = case["N"], case["Hkv"]
    if op == "keep":
        rows = 2 * B * H
        K = case["K"]
        return {"bytes": rows * (N * (dh * es + row) + (K + 1) * dh * es), "flops": rows * N * dh * 4}
    L = (case["L_lo"] + case["L_hi"]) / 2
    keys = L + N
    if case["window"]:
        keys = min(L, case["window"] + case["sinks"]) + N
    per_key = row if op == "packed" else dh * es
    return {"bytes": B * (2 * keys * H * per_key + 2 * N * case["Hq"] * dh * es),
            "flops": 4.0 * B * N * case["Hq"] * dh * keys}


# ------------------------------------------------- the definitions in 64 bits
def _exact_rows(x):
    """What the rows stand for, from the definition: the scale is the bf16
    number nearest to the fp32 quotient (it is stored), the rest in 64 bits."""
    x = x.double()
    lo = torch.minimum(x.min(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device=x.device))
    hi = torch.maximum(x.max(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device=x.device))
    scale = ((hi - lo).float().double() / 15).float().bfloat16().double()
    safe = torch.where(scale > 0, scale, 1.0)
    zero = (-lo / safe).round().clamp(0, 15)
    return scale * (((x / safe).round() + zero).clamp(0, 15) - zero)


def _exact_values(codes, par):
    low = torch.bitwise_and(codes, 15).double()
    high = torch.bitwise_right_shift(codes, 4).double()
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = low, high
    return par[..., 0, None].double() * (out - par[..., 1, None].double())


def exact(case, seed):
    st = prepare(case, seed)
    op, B, dh = case["op"], case["B"], case["dh"]
    if op == "pack":
        outs = []
        for x in (st["k"], st["v"]):
            full = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
            for b, n in enumerate(st["count"].tolist()):
                full[b, :n] = _exact_rows(x[b, :n])
            outs.append(full)
        return outs
    L = st["L"].tolist()
    if op == "keep":
        alen, nodes = st["alen"].tolist(), st["nodes"].tolist()
        new_len = torch.tensor([l + a + 1 for l, a in zip(L, alen)], dtype=torch.int32, device="cuda")
        outs = []
        for x in (st["k"], st["v"]):
            full = torch.zeros(B, case["K"] + 1, case["Hkv"], dh, dtype=torch.float64, device="cuda")
            for b in range(B):
                for j in range(alen[b] + 1):
                    full[b, j] = _exact_rows(x[b, nodes[b][j]])
            outs.append(full)
        return [new_len, *outs]
    N, H, G = case["N"], case["Hkv"], case["Hq"] // case["Hkv"]
    depth, anc = st["depth"].tolist(), st["anc"].tolist()
    out = torch.empty(B, N, case["Hq"], dh, dtype=torch.float64, device="cuda")
    for b in range(B):
        # additive mask, row by row
        bias = torch.full((N, L[b] + N), -math.inf, dtype=torch.float64, device="cuda")
        for n in range(N):
            seen = []
            first = 0 if case["window"] == 0 else max(0, L[b] + depth[n] - case["window"] + 1)
            bias[n, first:L[b]] = 0.0
            bias[n, :min(case["sinks"], L[b])] = 0.0
            for a in range(n + 1):
                p = L[b] + depth[a]
                if anc[n][a] and (p >= first or p < case["sinks"]):
                    seen.append(L[b] + a)
            bias[n, torch.tensor(seen, device="cuda")] = 0.0
        for h in range(H):
            if op == "packed":
                k, v = (_exact_values(st["cache"][i][b, h, :L[b] + N],
                                      st["cache"][i + 1][b, h, :L[b] + N]) for i in (0, 2))
            else:
                k, v = (st[x][b, :L[b] + N, h].double() for x in ("k", "v"))
            for g in range(G):
                s = st["q"][b, :, h * G + g].double() @ k.T / math.sqrt(dh) + bias
                out[b, :, h * G + g] = torch.softmax(s, dim=-1) @ v
    return out
