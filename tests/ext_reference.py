"""Plain 64-bit forms of the 4-bit cache and of windowed tree attention, and
the error bounds their kernels are held to.

Row format: the definition's fp32 steps are reproduced exactly.  A quotient
of two fp32 numbers computed in 64 bits and rounded once to 32 is the
correctly rounded fp32 quotient (53 >= 2 * 24 + 2), and rint of it is exact.

Attention bound, per output element (o exact, A = sum_j p_j |v_j| / sum_j p_j
the same average over |v|, S = max over visible j of scale * sum_d |q_d k_jd|):
  half a step of the output type                        eps_out * |o|
  the weights rounded once (c_p: fp16 2^-11, bf16 2^-8 plus the 1.5e-4 of the
  polynomial exponential; fp32 none) move o by at most  c_p * A
  and "fp16v", the kernel of more than 128 query rows per kv-head, rounds the
  decoded K and V to fp16 too: V is off by
  2^-11 of |v|, a score by 2^-11 S, in every weight of numerator and sum
                                                  (2^-10 + 2 * 2^-11 S) * A
  scores: a 128-term fp32 dot product is off by at most 128 * 2^-24 S = 2^-17 S,
  in every weight of the numerator and of the sum        2 * 2^-17 S * A
  fp32 sums, exponentials (2 ulp) and merges             2^-16 * A
  the range of the weights, for n visible keys with |v| <= v_max, relative to
  the row's largest weight (>= 1):
    fp32: a weight below 2^-126 may become 0             n * 2^-126 * v_max
    fp16: weight * value scale is held relative to a power of two R >= the
    largest scale s_max (R < 2 s_max) times 2^-7, in fp16, whose smallest step
    2^-24 is off by 2^-25 at most: 2^-25 * 2^-7 * R * 15 <= 2^-31 * 15 s_max a
    key, and s_max <= v_max as a row with a scale has a nonzero code
                                                         n * 2^-31 * 15 * v_max
The sum of these is the tolerance; no factor is fitted.
"""
from __future__ import annotations

import math

import torch

C_P = {"fp16": 2.0 ** -11, "fp16v": 2.0 ** -10, "bf16": 2.0 ** -8 + 1.5e-4, "fp32": 0.0}


def encode(x):
    """Rows x [..., dh] -> (codes uint8 [..., dh / 2], scale fp64, zero fp64 [...])."""
    x = x.double().cpu()
    lo = x.amin(-1).clamp(max=0.0)
    hi = x.amax(-1).clamp(min=0.0)
    rng = (hi - lo).float().double()
    scale = (rng / 15).float().bfloat16().double()
    bad = ~torch.isfinite(x).all(-1) | ~torch.isfinite(scale)
    scale = torch.where(bad, torch.full_like(scale, math.nan), scale)
    live = scale > 0
    div = torch.where(live, scale, torch.ones_like(scale))
    zero = (-lo / div).float().round().double().clamp(0, 15)
    c = (x / div[..., None]).float().round().double() + zero[..., None]
    c = torch.where(live[..., None], c.clamp(0, 15), torch.zeros_like(c)).to(torch.uint8)
    zero = torch.where(live, zero, torch.zeros_like(zero))
    return c[..., 0::2] | (c[..., 1::2] << 4), scale, zero


def decode(codes, par):
    """fp64 values of rows of codes (any device)."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    p = par.double()
    return p[..., 0:1] * (c - p[..., 1:2])


def tree_masks(plan):
    """(depth int64 [N], ancestor-or-self bool [N][N]) of an oracle tree plan."""
    N = len(plan["depth"])
    depth = torch.as_tensor(plan["depth"]).long()
    anc = torch.zeros(N, N, dtype=torch.bool)
    for i in range(N):
        j = i
        while j >= 0:
            anc[i, j] = True
            j = int(plan["parent"][j])
    return depth, anc


def visible(depth, anc, L, window, sinks):
    """bool [N][L + N]: slots each node sees."""
    N = depth.numel()
    vis = torch.zeros(N, L + N, dtype=torch.bool)
    for i in range(N):
        for p in range(L):
            vis[i, p] = window == 0 or p < sinks or p > L + int(depth[i]) - window
        for a in range(N):
            p = L + int(depth[a])
            vis[i, L + a] = bool(anc[i, a]) and (
                window == 0 or p < sinks or p > L + int(depth[i]) - window)
    return vis


def attention(q, k, v, Ls, plan, scale, window=0, sinks=0):
    """q [B][N][Hq][dh]; k, v [B][Hkv][Lcap][dh] fp64 values.  Returns (out,
    A, S, n v_max) fp64 on q's device; rows of a sequence that does not fit are 0.
    Values of slots a node does not see are not read."""
    B, N, Hq, dh = q.shape
    H, Lcap = k.shape[1], k.shape[2]
    G = Hq // H
    depth, anc = tree_masks(plan)
    out = torch.zeros(B, N, Hq, dh, dtype=torch.float64, device=q.device)
    A, S = torch.zeros_like(out), torch.zeros(B, N, Hq, 1, dtype=torch.float64, device=q.device)
    nv = torch.zeros_like(S)
    for b, L in enumerate(Ls):
        if L < 0 or L + N > Lcap:
            continue
        vis = visible_fast(depth, anc, L, window, sinks).to(q.device)
        seen = vis.any(0)
        kk = torch.where(seen[:, None], k[b, :, :L + N], 0.0)[:, None]   # [H][1][keys][dh]
        vv = torch.where(seen[:, None], v[b, :, :L + N], 0.0)[:, None]
        qq = q[b].double().view(N, H, G, dh).permute(1, 2, 0, 3)          # [H][G][N][dh]
        s = (qq @ kk.transpose(-1, -2)) * scale
        p = torch.softmax(s.masked_fill(~vis, -math.inf), -1)
        sa = ((qq.abs() @ kk.abs().transpose(-1, -2)) * scale).masked_fill(~vis, 0.0).amax(-1)

        def put(dst, x):
            dst[b].view(N, H, G, -1).copy_(x.permute(2, 0, 1, 3))
        put(out, p @ vv)
        put(A, p @ vv.abs())
        put(S, sa[..., None])
        put(nv, (vis.sum(-1)[None, None, :, None] * vv.abs().amax((-1, -2))[..., None, None])
            .expand(H, G, N, 1).double())
    return out, A, S, nv


def visible_fast(depth, anc, L, window, sinks):
    N = depth.numel()
    pos = torch.cat([torch.arange(L), L + depth])
    vis = torch.cat([torch.ones(N, L, dtype=torch.bool), anc], 1)
    if window:
        vis &= (pos[None] < sinks) | (pos[None] > L + depth[:, None] - window)
    return vis


def assert_close(got, ref, A, S, nv, dtype, weights, what=""):
    half = torch.finfo(dtype).eps / 2
    floor = 15 * 2.0 ** -31 if weights.startswith("fp16") else 2.0 ** -126
    score = 2.0 ** -17 + (2.0 ** -11 if weights == "fp16v" else 0.0)
    tol = half * ref.abs() + A * (C_P[weights] + 2 * score * S + 2.0 ** -16) + floor * nv
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst excess "
        f"{float((err / tol.clamp(min=1e-300)).nan_to_num(nan=math.inf).max()):.3g} x")
