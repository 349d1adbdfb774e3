"""float64 attention over a mask of visible keys, with error bounds that follow
each row's own weights, so that they shrink with the output as lists grow.

With weights w_k = exp(x_k) / sum exp(x) and |dx_k| the error of a score,
O' - O = sum_k w_k (exp(dx_k) - 1) (v_k - O), so to first order
|dO| <= sum_k w_k |dx_k| |v_k - O|.  Scores: a float32 sum of D products and two
more roundings, (D + 4) u sum_d |q_d k_d| scale with u = 2^-24, the roundings of
the scaled value and of its difference to the reference, u (2 |x| + 2 |x - top|),
and a base-2 exponential of 2^-22.  (A mask of 2^28 or more absorbs its score, as
the float32 sum does.)  The float32 sums over keys run through about n / 16 steps, each
of which a tensor-core product may truncate: (16 + n / 8) u sum w |v|.  A
probability that enters its product rounded adds p_rel of itself and p_abs of the
row's largest one: `single` is one value of the element type, `halves` two (16
bits of bf16; of f16 21 bits and what lies under its smallest value, see the
kernels), float32 none.  Last, the output's own rounding.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
ABSORBS = 2.0 ** 28   # a mask whose float32 spacing is 32
LOW = torch.finfo(torch.float32).min
HALF = {torch.float32: U32, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def mask_kinds(g, *shape):
    """Masks [..., keys] with a kind a row: all lowest; lowest and -inf; two values below -2.4e38; one at zero among
    lowest; ordinary ones; all -inf; all -1e9; some 1e9 among ordinary ones."""
    rows, keys = shape[:-1], shape[-1]
    m = torch.full(shape, LOW, device="cuda")
    kind = torch.randint(0, 8, rows, generator=g, device="cuda")[..., None]
    r = torch.rand(shape, generator=g, device="cuda")
    m = torch.where((kind == 1) & (r < 0.5), -math.inf, m)
    m = torch.where((kind == 2) & (r < 0.3), -3.0e38, m)
    m = torch.where((kind == 3) & (torch.arange(keys, device="cuda") == 2), 0.0, m)
    m = torch.where(kind == 4, r, m)
    m = torch.where(kind == 6, -1e9, m)
    m = torch.where(kind == 7, torch.where(r < 0.2, 1e9, r), m)
    return torch.where(kind == 5, -math.inf, m)


def p_error(dt, how):
    """(relative, relative to the row's largest probability) error of a probability."""
    if dt == torch.float32:
        return 0.0, 0.0
    if how == "single":
        return HALF[dt], 0.0 if dt == torch.bfloat16 else 2.0 ** -30   # half f16's least value, 2^-25, on a top of 2^5
    return (2.0 ** -15, 0.0) if dt == torch.bfloat16 else (2.0 ** -20, 2.0 ** -34)


def attention(q, k, v, vis, *, p="halves", scale=0.0, mask=None, softcap=0.0, sink=None, zero=True, kv_scales=None,
              extra_score=0.0):
    """q [B, H, Sq, D], k and v [B, G, Sk, D] in storage types, vis bool [B, Sq, Sk], on any device
    -> O, LSE, bound of O, bound of LSE.  extra_score: relative error of each product q_d k_d beyond float32's."""
    dt, dev = q.dtype, q.device
    B, H, Sq, D = q.shape
    per = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    if kv_scales is not None:
        ks, vs = (s.double().view(1, -1, 1, D) if s.numel() > 1 else s.double() for s in kv_scales)
        k, v = k * ks, v * vs
    live = vis.any(1)[:, None, :, None]
    k = torch.where(live, k, 0.0).repeat_interleave(per, 1)
    v = torch.where(live, v, 0.0).repeat_interleave(per, 1)
    scale = scale or 1 / math.sqrt(D)
    x = q @ k.transpose(-1, -2) * scale
    mag = q.abs() @ k.abs().transpose(-1, -2) * abs(scale)
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    if mask is not None:
        x = torch.where(mask.abs() >= ABSORBS, mask.double(), x + mask.double())
    x = x.masked_fill(~vis[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    sg = torch.full((B, H, Sq, 1), -math.inf, dtype=torch.float64, device=dev)
    if sink is not None:
        sg = sink.double().view(1, H, 1, 1).expand(B, H, Sq, 1)
        top = torch.maximum(top, sg)
    base = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(x - base)
    den = e.sum(-1, keepdim=True) + torch.exp(sg - base)
    w = e / torch.where(den == 0, 1.0, den)
    o = w @ v
    lse = (base + torch.log(den)).squeeze(-1)
    # bounds
    size = torch.where(x.abs() < ABSORBS, x.abs(), 0.0)
    away = torch.where(x > -math.inf, (x - base).abs(), 0.0).clamp(max=200)
    dx = (D + 4) * U32 * mag + extra_score * mag + U32 * (2 * size + 2 * away) + 2.0 ** -22
    if softcap:
        dx = dx + softcap * 2.0 ** -21
    wd = w * dx
    n = vis.sum(-1).view(B, 1, Sq, 1).double()
    va = v.abs()
    steps = (16 + n / 8) * U32
    rel, floor = p_error(dt, p)
    spread = wd @ va + wd.sum(-1, keepdim=True) * o.abs()
    tol = 1.01 * spread + (2 * steps + rel) * (w @ va) + steps * o.abs()
    seen = vis[:, None].double()
    tol = tol + 2 * floor * w.amax(-1, keepdim=True) * (seen @ va)
    tol = tol + HALF[dt] * o.abs() + 2.0 ** -25
    tol_l = (1.01 * wd.sum(-1, keepdim=True) + steps).squeeze(-1) + lse.abs() * 2.0 ** -22 + 2.0 ** -22
    none = den == 0
    o = torch.where(none, 0.0 if zero else math.nan, o)
    lse = torch.where(none.squeeze(-1), -math.inf, lse)
    return o, lse, tol, tol_l


def worst(got, ref, tol):
    """Largest |got - ref| / tol; NaN and infinities have to agree."""
    got = got.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaN pattern"
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], ref[inf]), "infinities"
    ok = ~inf & ~torch.isnan(ref)
    r = ((got - ref).abs() / tol.expand_as(ref))[ok]
    return float(r.max()) if r.numel() else 0.0


def check(got, ref, tol, where=""):
    r = worst(got, ref, tol)
    assert r <= 1, f"{where}: {r:.3g} times the bound"


def rows_of(pool, table, ps, rows, nhd=False):
    """[B, G, rows, D]: the rows that the page lists name (every list value has to name a page)."""
    r = torch.arange(rows, device=pool.device)
    page = table[:, r // ps].long()
    return (pool[page, r % ps] if nhd else pool[page, :, r % ps]).transpose(1, 2)
