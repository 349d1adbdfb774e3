"""float64 references of the serving operators (windows with first keys, paged
caches, Q/K norm and rotation), in plain numpy-style torch on the CPU, with the
error bounds that the tests hold the kernels to.

Bounds (u = 2^-24, the float32 half step; U = the half step of the element
type, 0 for float32).  A score is a float32 sum of D products and two more
roundings, so |ds| <= (D + 4) u sum_d |q_d k_d| scale, plus the type's
half step on each product where Q is rounded again (int8 caches: 2^-11).  A
probability then has a relative error of at most 2 |ds| + 2^-20 (a base-2
exponential of 2^-22, its argument rounded at |x| <= 2^6).  The sums over n
keys add n u, and P rounded to the element type U.  With |v| <= V:
|dO| <= V (4 ds + 2^-19 + 2 n u + U + n 2^-25) + U |O| (the last for the
output's rounding, n 2^-25 for f16 probabilities below its normal range)."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
HALF = {torch.float32: U32, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def visible(q_len, k_len, lens, *, causal=True, offset=None, window=-1, first=0, seg=None):
    """bool [B, q_len, k_len].  offset None: right-aligned to each entry's length."""
    n = torch.as_tensor(lens).view(-1, 1, 1).clamp(0, k_len)
    i, k = torch.arange(q_len).view(1, -1, 1), torch.arange(k_len).view(1, 1, -1)
    vis = (k < n).expand(n.shape[0], q_len, k_len)
    if causal:
        diag = i + (n - q_len if offset is None else offset)
        s = torch.zeros_like(diag) if seg is None else seg.clamp(0, k_len).unsqueeze(-1)
        vis = vis & (k <= diag) & (k >= s)
        if window >= 0:
            vis = vis & ((k >= diag - window) | (k < s + first))
    return vis


def attention(q, k, v, vis, *, scale=0.0, mask=None, softcap=0.0, sink=None, zero=True, kv_scales=None, half_q=False):
    """q [B, H, Sq, D], k and v [B, G, Sk, D] (storage types), vis [B, Sq, Sk] -> (O, LSE, |dO| bound, |dLSE| bound)."""
    dt = q.dtype
    B, H, Sq, D = q.shape
    per = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    if kv_scales is not None:   # per (kv head, channel) or one
        ks, vs = (s.double().view(1, -1, 1, D) if s.numel() > 1 else s.double() for s in kv_scales)
        k, v = k * ks, v * vs
    live = vis.any(1)   # values of keys no row sees may be anything
    k = torch.where(live[:, None, :, None], k, 0.0).repeat_interleave(per, 1)
    v = torch.where(live[:, None, :, None], v, 0.0).repeat_interleave(per, 1)
    scale = scale or 1 / math.sqrt(D)
    s = q @ k.transpose(-1, -2) * scale
    mag = q.abs() @ k.abs().transpose(-1, -2) * abs(scale)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    x = s if mask is None else s + mask.double()
    x = x.masked_fill(~vis[:, None], -math.inf)
    seen = vis[:, None] & (x != -math.inf)
    top = x.amax(-1, keepdim=True) if x.shape[-1] else torch.full_like(x.sum(-1, keepdim=True), -math.inf)
    sg = torch.full((B, H, Sq, 1), -math.inf, dtype=torch.float64)
    if sink is not None:
        sg = sink.double().view(1, H, 1, 1).expand(B, H, Sq, 1)
        top = torch.maximum(top, sg)
    base = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(x - base)
    den = p.sum(-1, keepdim=True) + torch.exp(sg - base)
    bad = torch.isnan(x).any(-1, keepdim=True) | (x == math.inf).any(-1, keepdim=True)
    o = torch.where(den == 0, 0.0 if zero else math.nan, p @ v / den)
    o = torch.where(bad, math.nan, o)
    lse = torch.where(bad, math.nan, base + torch.log(den)).squeeze(-1)
    # bounds
    z = torch.zeros((), dtype=torch.float64)
    ds = (D + 4) * U32 * torch.where(seen, mag, z).amax(-1, keepdim=True) if x.shape[-1] else z
    if half_q:
        ds = ds + 2.0 ** -11 * torch.where(seen, mag, z).amax(-1, keepdim=True)
    ds = ds + 2.0 ** -22 * torch.where(seen, x.abs(), z).amax(-1, keepdim=True) if x.shape[-1] else ds
    if softcap:
        ds = ds + softcap * 2.0 ** -21
    n = seen.sum(-1, keepdim=True)
    # int8 codes: the value is code * scale, and the biased integers of that pass sum to at most 1279 / 127 as much
    big = 11.0 if kv_scales is not None else 1.0
    vmax = v.abs().amax((-1, -2), keepdim=True) if x.shape[-1] else z
    U = HALF[dt]
    up = 0.0 if dt == torch.float32 else max(U, 2.0 ** -11 * big if kv_scales is not None else 0.0)
    tol = vmax * (4 * ds + 2.0 ** -19 + 2 * n * U32 * big + up + n * 2.0 ** -25) + U * o.abs() + 2.0 ** -25
    tol_l = (2 * ds + 2.0 ** -19 + n * U32).squeeze(-1) + lse.abs() * 2.0 ** -21
    if kv_scales is not None:   # sums of probabilities rounded to f16
        tol_l = tol_l + 2.0 ** -11
    return o, lse, tol, tol_l


def check(got, ref, tol, where=""):
    """Element by element: the same NaN and infinity pattern, and |got - ref| <= tol elsewhere."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{where}: NaN pattern"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]) and not torch.isinf(got[~inf]).any(), f"{where}: infinities"
    d = (got - ref).abs()
    over = ~(d <= tol.expand_as(ref)) & ~inf & ~torch.isnan(ref)
    assert not over.any(), (f"{where}: {int(over.sum())} of {over.numel()} beyond the bound; worst "
                            f"{(d / tol.expand_as(ref))[over].max():.3g} times, first at {over.nonzero()[0].tolist()}")


def gather(pool, table, ps, rows, nhd):
    """The rows [B, G, rows, D] that the lists name and whether each has a page, bool [B, rows]."""
    r = torch.arange(rows)
    page = table[:, r // ps].long()
    ok = (page >= 0) & (page < pool.shape[0])
    page = torch.where(ok, page, 0)
    if pool.shape[0] == 0:
        raise ValueError("empty pool")
    x = pool[page, r % ps] if nhd else pool[page, :, r % ps]   # [B, rows, G, D]
    return x.transpose(1, 2), ok


def prep(x, w, cos, sin, pos, *, eps, norm, rot, inter):
    """Norm and rotation of x [B, S, N, D] in float64, and the |d| bound of a float32 evaluation before its rounding.

    With y the normed value: sum of squares D u / 2 relative (a square root halves it), division, two
    products: (D / 2 + 5) u; the rotation adds two products and a sum: 3 u of |ya cos| + |yc sin|."""
    D = x.shape[-1]
    y = x.double()
    if norm:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w.double()
    mag = y.abs()
    if rot:
        c, s = cos.double()[pos].unsqueeze(2), sin.double()[pos].unsqueeze(2)
        h = rot // 2
        ia = torch.arange(0, rot, 2) if inter else torch.arange(h)
        ic = ia + 1 if inter else ia + h
        a, b = y[..., ia], y[..., ic]
        z, m = y.clone(), mag.clone()
        z[..., ia], z[..., ic] = a * c - b * s, b * c + a * s
        m[..., ia], m[..., ic] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
        y, mag = z, m
    return y, (D / 2 + 8) * U32 * mag
