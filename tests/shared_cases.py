"""Inputs of attn_fwd_shared and their float64 results under the bounds of
serving_bounds.py: every pool row that no row of its entry (of the batch, in the
prefix) sees holds NaN."""
from __future__ import annotations

import torch

import serving_bounds as sb
from attention_attn_fwd_02_gb300 import attn

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(dt, D, B, Sq, H, G, ps, prefix, lens, seed, *, nhd=False, i8=None, max_rows=None, causal=True, offset=None,
         mask=None, holes=(), prefix_holes=(), pad=0, bhsd=False, poison=True, **kw):
    """lens: own keys of each entry.  holes: (entry, page) of lists, and pages of the prefix's list, that name no
    page.  pad: extra elements between the rows of the pools and of q.  i8: 'tensor' or 'channel'."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = DT[dt]
    cap = max(lens) if max_rows is None else max_rows
    width, pw = -(-cap // ps), -(-prefix // ps)
    n_pages = B * width + pw + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table, ptab = perm[:B * width].view(B, width).clone(), perm[B * width:B * width + pw].clone()
    for b, j in holes:
        table[b, j] = (-1, n_pages, 2 ** 31 - 1)[(b + j) % 3]
    for j in prefix_holes:
        ptab[j] = (-1, n_pages, -2 ** 31)[j % 3]
    shape = (n_pages, ps, G, D + pad) if nhd else (n_pages, G, ps, D + pad)

    def pool():
        if i8:
            return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)[..., :D]
        return torch.randn(shape, generator=g, device="cuda").to(T)[..., :D]

    k, v = pool(), pool()
    scales = [torch.rand(G * D if i8 == "channel" else 1, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2)] \
        if i8 else None
    q = torch.randn(B, Sq, H, D + pad, generator=g, device="cuda").to(T)[..., :D]
    if bhsd:
        q = q.transpose(1, 2).contiguous().transpose(1, 2)
    n = torch.tensor(lens, device="cuda").clamp(0, cap)
    own = torch.arange(cap, device="cuda")
    vis = (own < n.view(B, 1, 1)).expand(B, Sq, cap)
    if causal:
        diag = torch.arange(Sq, device="cuda").view(1, -1, 1) + (n.view(B, 1, 1) - Sq if offset is None else offset)
        vis = vis & (own <= diag)
    vis = torch.cat([torch.ones(B, Sq, prefix, dtype=torch.bool, device="cuda"), vis], 2)

    def named(t, rows):   # (page, row in it) of each row of lists t, and whether the list names a page
        r = torch.arange(rows, device="cuda")
        page = t[:, r // ps].long() if rows else t[:, :0].long()
        return page, r % ps, (page >= 0) & (page < n_pages)

    pp, pr, pok = named(ptab[None], prefix)
    op, orow, ook = named(table, cap)
    vis = vis & torch.cat([pok.expand(B, prefix), ook], 1)[:, None]

    def rows_of(p):
        take = lambda page, r, ok: torch.where(ok[..., None, None], p[page.clamp(0, n_pages - 1), r] if nhd else  # noqa: E731
                                               p[page.clamp(0, n_pages - 1), :, r], 0)
        return torch.cat([take(pp, pr, pok).expand(B, -1, -1, -1), take(op, orow, ook)], 1).transpose(1, 2)

    kk, vv = rows_of(k), rows_of(v)
    if poison and not i8:
        seen = torch.zeros(n_pages, ps, dtype=torch.bool, device="cuda")
        live = vis.any(1)
        seen[pp[0][live[:, :prefix].any(0)], pr[live[:, :prefix].any(0)]] = True
        for b in range(B):
            at = live[b, prefix:]
            seen[op[b][at], orow[at]] = True
        for t in (k, v):
            (t if nhd else t.transpose(1, 2))[~seen] = float("nan")
    args = dict(k_lens=n.to(torch.int32), page_layout="nhd" if nhd else "hnd", causal=causal, causal_offset=offset,
                max_rows=cap, mask=mask, **kw)
    if i8:
        args.update(k_scale=scales[0], v_scale=scales[1])
    ref_kw = dict(mask=None if mask is None else mask[..., :prefix + cap].expand(B, H, Sq, -1),
                  softcap=kw.get("softcap", 0.0), scale=kw.get("scale", 0.0), kv_scales=scales,
                  zero=kw.get("masked_rows") == "zero",
                  sink=kw["head_sink"] if kw.get("head_sink") is not None else
                  torch.zeros(H, device="cuda") if kw.get("smooth_softmax") else None)
    return dict(call=(q, k, v, ptab, prefix, table), args=args, ref=(q.transpose(1, 2), kk, vv, vis), ref_kw=ref_kw)


def run(c, **kw):
    return attn.fwd_shared(*c["call"], **dict(c["args"], **kw))


def check(c, out, lse=None, where="", **kw):
    o, l, tol, tol_l = sb.attention(*c["ref"], p="single", **dict(c["ref_kw"], **kw))
    sb.check(out.transpose(1, 2), o, tol, where)
    if lse is not None:
        sb.check(lse, l, tol_l, where + " lse")
