"""Cases of two operators for requests that ask about one long image, video or document, with plain forms.

* ``axes``    the step before attention with positions on several axes (time, height, width): per-head
              RMS norm of Q and K, rotation in which every pair of elements takes its angle at its own
              axis's position, and the write of K and V into the cache (``attn_qkv_prep_axes``);
* ``shared``  attention of a batch whose entries share a prefix: the queries of every entry, one token or
              many, see the prefix's keys and, causally, their entry's own keys, all in one paged cache
              (``attn_fwd_shared``).

``run`` computes a case in its plain form (elementary torch operations in float32, rounded once at
the end), or with ``own`` set through the library's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------------


def listed():
    shared = dict(op="shared", q=1, nhd=False)
    axes = dict(op="axes", ps=64, inter=False, by="sections")
    return [
        # four questions on a short prompt, the next token of each: a call's latency
        dict(shared, name="shared_four_short", dtype="bf16", B=4, H=32, G=8, D=128, ps=16, prefix=1000, min_own=1,
             max_own=100),
        # a full serving batch behind one long instruction
        dict(shared, name="shared_batch64", dtype="bf16", B=64, H=32, G=8, D=128, ps=64, prefix=8192, min_own=1,
             max_own=1024),
        # many questions about one very long document
        dict(shared, name="shared_long", dtype="bf16", B=32, H=32, G=8, D=128, ps=64, prefix=131072, min_own=1,
             max_own=512),
        # hundreds of samples of one prompt, some not yet begun
        dict(shared, name="shared_many", dtype="f16", B=200, H=12, G=4, D=64, ps=16, nhd=True, prefix=2003, min_own=0,
             max_own=400),
        # a few drafted tokens of each sample
        dict(shared, name="shared_drafts", dtype="bf16", B=16, q=5, H=32, G=8, D=128, ps=32, prefix=20011, min_own=5,
             max_own=700),
        # the questions' own prompts, behind a long document
        dict(shared, name="shared_questions", dtype="bf16", B=8, q=200, H=32, G=8, D=128, ps=64, prefix=16384,
             min_own=200, max_own=1000),
        # long prompts behind an instruction
        dict(shared, name="shared_prompts", dtype="f16", B=3, q=2048, H=16, G=2, D=128, ps=128, prefix=4099,
             min_own=2048, max_own=2048, nhd=True),
        # a small float32 model
        dict(shared, name="shared_small_f32", dtype="f32", B=5, q=33, H=12, G=4, D=64, ps=16, prefix=501, min_own=33,
             max_own=100),
        # the step of a serving batch: one token a sequence
        dict(axes, name="axes_step", dtype="bf16", B=64, S=1, H=32, G=8, D=128, rot=128, axes=3, grid="1x1x1",
             cap=256, min_len=1),
        # a video's tokens into a paged cache
        dict(axes, name="axes_video", dtype="bf16", B=1, S=16384, H=32, G=8, D=128, rot=128, axes=3, grid="16x30x34",
             cap=16384, min_len=16384),
        # images and text, axes in turn from pair to pair, a ragged batch
        dict(axes, name="axes_in_turn", dtype="f16", B=2, S=5003, H=12, G=4, D=64, rot=64, axes=3, by="turns",
             grid="3x37x41", cap=5100, ps=16, min_len=4000),
        # an image encoder's layer, height and width, a contiguous cache, float32
        dict(axes, name="axes_image_f32", dtype="f32", B=3, S=1369, H=12, G=12, D=64, rot=64, axes=2, grid="37x37",
             cap=1369, ps=0, min_len=1369),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "axes"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while True:
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4, 8])
        if op == "shared":
            c = dict(op=op, dtype=dtype, B=_log(rng, 1, 256), q=1 if rng.random() < 0.5 else _log(rng, 2, 2048), H=H,
                     G=G, D=rng.choice([64, 128]), ps=rng.choice([8, 16, 24, 32, 64, 128]),
                     prefix=_log(rng, 64, 131072), nhd=rng.random() < 0.5)
            c["max_own"] = c["q"] + _log(rng, 1, 2048)
            c["min_own"] = rng.randint(min(c["q"], 5) - 1, c["max_own"])
            pairs = c["B"] * H * c["q"] * (c["prefix"] + c["max_own"])
            if pairs <= 2 ** 30 and work(c)["flops"] <= (4e11 if dtype != "f32" else 2e10) and \
                    work(c)["bytes"] <= 6e8 and c["B"] * c["max_own"] <= 2 ** 17:
                return c
        else:
            D = rng.choice([64, 128, 256])
            n = rng.choice([2, 3, 3])
            c = dict(op=op, dtype=dtype, B=_log(rng, 1, 96), S=1 if rng.random() < 0.3 else _log(rng, 2, 16384), H=H,
                     G=G, D=D, rot=rng.choice([D, D, D // 2]), axes=n, by=rng.choice(["sections", "sections", "turns"]),
                     inter=rng.random() < 0.25, ps=rng.choice([0, 16, 24, 64]))
            c["grid"] = "x".join(str(rng.randint(1, 1 + int(c["S"] ** (1 / n)))) for _ in range(n))
            c["cap"] = c["S"] + rng.randint(0, 256)
            c["min_len"] = rng.randint(1, c["S"])
            if work(c)["bytes"] <= 5e8 and c["B"] * c["cap"] * G * D <= 2 ** 25:
                return c


def _lens(c):
    """Own keys (shared) or real tokens (axes) of each batch entry."""
    lo, hi = (c["min_own"], c["max_own"]) if c["op"] == "shared" else (c["min_len"], c["S"])
    r = random.Random(c["B"] * 7919 + lo)
    got = [r.randint(lo, hi) for _ in range(c["B"])]
    got[0], got[-1] = lo, hi   # both ends occur
    return got


def _sections(c):
    """The axis of each rotated pair: a stretch of pairs an axis (the first the shortest), or axes in turn."""
    half, n = c["rot"] // 2, c["axes"]
    if c["by"] == "turns":
        return [j % n for j in range(half)]
    first = half // n if n == 2 else half // 4
    rest = (half - first) // (n - 1)
    return [0 if j < first else min(n - 1, 1 + (j - first) // rest) for j in range(half)]


def work(c):
    B, H, G, D, es = c["B"], c["H"], c["G"], c["D"], 4 if c["dtype"] == "f32" else 2
    lens = _lens(c)
    if c["op"] == "shared":
        q, rows = c["q"], [c["prefix"]] + lens
        pairs = B * q * c["prefix"] + sum(min(max(n - q + i + 1, 0), n) for n in lens for i in range(q))
        return {"bytes": 2 * sum(rows) * G * D * es + 2 * B * q * H * D * es + 4 * sum(-(-n // c["ps"]) for n in rows),
                "flops": 4 * pairs * H * D}
    tokens, real = B * c["S"], sum(lens)
    values = 2 * tokens * H * D + 4 * real * G * D + 2 * D
    return {"bytes": values * es + 4 * c["rot"] * min(tokens, c["cap"]) + 4 * (c["axes"] + 1) * tokens,
            "flops": (tokens * H + real * G) * (4 * D + 3 * c["rot"])}


# ---- inputs --------------------------------------------------------------------------------------


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, H, G, D, dt, ps = c["B"], c["H"], c["G"], c["D"], DTYPES[c["dtype"]], c["ps"]
    lens = _lens(c)
    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}

    def lists(counts, width):
        """Page lists: the pages of a pool in random order, -1 where an entry holds no page."""
        perm = torch.randperm(max(sum(counts), 1), generator=g, device=DEV).to(torch.int32)
        table = torch.full((len(counts), max(width, 1)), -1, dtype=torch.int32, device=DEV)
        have = torch.arange(table.shape[1], device=DEV) < torch.tensor(counts, device=DEV)[:, None]
        table[have] = perm[:sum(counts)]
        return table, perm.numel()

    if c["op"] == "shared":
        n_own, n_pre = -(-c["max_own"] // ps), -(-c["prefix"] // ps)
        both, n_pages = lists([-(-n // ps) for n in lens] + [n_pre], max(n_own, n_pre))
        s["table"], s["prefix"] = both[:-1, :n_own].contiguous(), both[-1, :n_pre].contiguous()
        shape = (n_pages, ps, G, D) if c["nhd"] else (n_pages, G, ps, D)
        s["k"], s["v"] = (torch.randn(shape, generator=g, device=DEV, dtype=dt) for _ in range(2))
        s["q"] = torch.randn(B, c["q"], H, D, generator=g, device=DEV).to(dt)
        s["out"] = torch.empty_like(s["q"])
    else:
        S, cap = c["S"], c["cap"]
        qkv = (1.5 * torch.randn(B, S, H + 2 * G, D, generator=g, device=DEV)).to(dt)   # a packed projection
        s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + G], qkv[:, :, H + G:]
        s["qw"], s["kw"] = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt) for _ in range(2))
        i = torch.arange(S, device=DEV)[None]
        n = s["lens"][:, None]
        past = torch.randint(0, 1 << 30, (B, 1), generator=g, device=DEV) % (cap - n + 1)
        s["row"] = torch.where(i < n, past + i, -1).to(torch.int32)
        # The first tokens are a grid of patches; text follows with one position on every axis.
        extents = [int(x) for x in c["grid"].split("x")]
        size = math.prod(extents)
        at, grid = torch.arange(S, device=DEV), []
        for extent in reversed(extents):
            grid.insert(0, at % extent)
            at = at // extent
        text = max(extents) + torch.arange(S, device=DEV) - size
        pos = torch.stack([torch.where(torch.arange(S, device=DEV) < size, x, text) for x in grid])[:, None]
        s["pos"] = torch.where(i < n, (past + pos) % cap, 0).to(torch.int32).contiguous()   # [axes, B, S]
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        ang = torch.arange(cap, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["table"], n_pages = lists([-(-cap // ps)] * B, -(-cap // ps)) if ps else (None, B)
        shape = (n_pages, G, ps or cap, D)
        s["kc"], s["vc"] = torch.zeros(shape, dtype=dt, device=DEV), torch.zeros(shape, dtype=dt, device=DEV)
        s["out"] = torch.empty(B, S, H, D, dtype=dt, device=DEV)
    if own:
        _plan(s)
    return s


# ---- the library's entry points ------------------------------------------------------------------


def _plan(s):
    """The problem description and workspace that a program keeps from call to call."""
    from attention_attn_fwd_02_gb300 import attn

    c = s["case"]
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    s["attn"] = attn
    strides = lambda t, row, head: (0, t.stride(0), t.stride(head), t.stride(row))  # noqa: E731
    if c["op"] == "axes":
        s["pages"] = attn.make_pages(c["ps"], s["kc"].shape[0], s["table"].data_ptr(), s["table"].stride(0)) \
            if c["ps"] else None
        s["axes"] = attn.make_axes(_sections(c), s["pos"].stride(0))
        s["plan"] = attn.make_prep(dict(
            batch=B, seq_len=c["S"], heads=H, kv_heads=G, head_dim=D, rot_dim=c["rot"], dtype=c["dtype"],
            interleaved=c["inter"], norm=True, eps=1e-6, max_pos=c["cap"], cache_rows=c["cap"],
            q_layout=strides(s["q"], 1, 2), k_layout=strides(s["k"], 1, 2), v_layout=strides(s["v"], 1, 2),
            q_out_layout=strides(s["out"], 1, 2), k_out_layout=strides(s["kc"], 2, 1),
            v_out_layout=strides(s["vc"], 2, 1)))
        return
    row, head = (1, 2) if c["nhd"] else (2, 1)
    s["plan"] = attn.make_problem(dict(
        batch=B, heads=H, kv_heads=G, head_dim=D, dtype=c["dtype"], q_len=c["q"], k_len=c["max_own"], causal=True,
        causal_align="klens", masked_rows="zero", q_layout=strides(s["q"], 1, 2), o_layout=strides(s["out"], 1, 2),
        k_layout=strides(s["k"], row, head), v_layout=strides(s["v"], row, head)))
    s["pages"] = attn.make_pages(c["ps"], s["k"].shape[0], s["table"].data_ptr(), s["table"].stride(0))
    s["pre"] = attn.make_prefix(c["prefix"], s["prefix"].data_ptr())
    size = attn.attn_fwd_shared_workspace_size(s["plan"], s["pages"], s["pre"])
    s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)


def _own(s):
    c, attn, st = s["case"], s["attn"], torch.cuda.current_stream().cuda_stream
    ptr = torch.Tensor.data_ptr
    if c["op"] == "shared":
        rc = attn.attn_fwd_shared(s["plan"], s["pages"], s["pre"], ptr(s["q"]), ptr(s["k"]), ptr(s["v"]),
                                  ptr(s["out"]), None, ptr(s["lens"]), None, ptr(s["ws"]), s["ws"].numel(), st)
    else:
        rc = attn.attn_qkv_prep_axes(s["plan"], s["pages"], s["axes"], ptr(s["q"]), ptr(s["k"]), ptr(s["v"]),
                                     ptr(s["qw"]), ptr(s["kw"]), ptr(s["cos"]), ptr(s["sin"]), ptr(s["pos"]),
                                     ptr(s["row"]), ptr(s["out"]), ptr(s["kc"]), ptr(s["vc"]), st)
    if rc:
        raise attn.AttnError(rc, c["op"])
    return {"q": s["out"], "k": s["kc"], "v": s["vc"]} if c["op"] == "axes" else {"o": s["out"]}


# ---- the plain forms -----------------------------------------------------------------------------


def _shared(s):
    c = s["case"]
    B, q, H, G, D, P = c["B"], c["q"], c["H"], c["G"], c["D"], c["prefix"]
    per = H // G

    def rows(pool, table):   # [entries, G, keys, D] in float32
        x = pool[table.clamp(min=0).long()]
        return (x.permute(0, 3, 1, 2, 4) if c["nhd"] else x.permute(0, 2, 1, 3, 4)).reshape(len(table), G, -1, D).float()

    pk, pv = (rows(t, s["prefix"][None])[0, :, :P] for t in (s["k"], s["v"]))
    ok, ov = (rows(t, s["table"]) for t in (s["k"], s["v"]))
    queries = s["q"].float().view(B, q, G, per, D).permute(2, 0, 1, 3, 4) * (1 / math.sqrt(D))   # [G, B, q, per, D]
    flat = queries.reshape(G, B * q * per, D)
    xp = torch.matmul(flat, pk.transpose(-1, -2)).view(G, B, q * per, P)
    xo = torch.matmul(queries.reshape(G, B, q * per, D), ok.permute(1, 0, 3, 2))
    key = torch.arange(ok.shape[2], device=DEV)
    n = s["lens"].view(B, 1, 1)
    diag = torch.arange(q, device=DEV).repeat_interleave(per).view(1, -1, 1) + n - q
    xo = xo.masked_fill(~((key < n) & (key <= diag)), -math.inf)
    m = torch.maximum(xp.amax(-1, keepdim=True), xo.amax(-1, keepdim=True))
    xp, xo = torch.exp(xp - m), torch.exp(xo - m)
    o = torch.matmul(xp.view(G, -1, P), pv).view(G, B, q * per, D) + torch.matmul(xo, ov.transpose(0, 1))
    o = o / (xp.sum(-1, keepdim=True) + xo.sum(-1, keepdim=True))
    return {"o": o.view(G, B, q, per, D).permute(1, 2, 0, 3, 4).reshape(B, q, H, D).to(s["q"].dtype)}


def _rotated(x, w, cos, sin, c):
    """RMS norm over the head, times its weight, and the rotation of the first `rot` elements."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _axes(s):
    c = s["case"]
    axis = torch.tensor(_sections(c), device=DEV)
    pos = s["pos"].long()[axis].permute(1, 2, 0)   # [B, S, pairs]: each pair's own position
    pair = torch.arange(len(axis), device=DEV)
    cos, sin = s["cos"][pos, pair].unsqueeze(2), s["sin"][pos, pair].unsqueeze(2)
    dt = s["out"].dtype
    q = _rotated(s["q"], s["qw"], cos, sin, c).to(dt)
    k = _rotated(s["k"], s["kw"], cos, sin, c).to(dt)
    b, i = torch.nonzero(s["row"] >= 0, as_tuple=True)
    row = s["row"][b, i].long()
    ps = s["kc"].shape[2]
    page = s["table"][b, row // ps].long() if c["ps"] else b
    s["kc"].transpose(1, 2)[page, row % ps] = k[b, i]
    s["vc"].transpose(1, 2)[page, row % ps] = s["v"][b, i]
    return {"q": q, "k": s["kc"], "v": s["vc"]}


def run(s):
    if own:
        return _own(s)
    return {"shared": _shared, "axes": _axes}[s["case"]["op"]](s)


# ---- 64 bits, from the definitions -----------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    per, ps = H // G, c["ps"]
    lens = _lens(c)
    f8 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "shared":
        q, P = c["q"], c["prefix"]
        out = torch.zeros(B, q, H, D, **f8)

        def take(pool, table, n, g):   # the first n rows of a page list, of one kv head
            r = torch.arange(n, device=DEV)
            page, at = table.long()[r // ps], r % ps
            return (pool[page, at, g] if c["nhd"] else pool[page, g, at]).double()

        for g in range(G):
            pk, pv = (take(s[x], s["prefix"], P, g) for x in "kv")
            for b, n in enumerate(lens):
                k, v = (torch.cat([p, take(s[x], s["table"][b], n, g)]) for p, x in ((pk, "k"), (pv, "v")))
                # query i is the entry's token n - q + i
                late = torch.arange(P + n, device=DEV)[None] - P - (torch.arange(q, device=DEV)[:, None] + n - q) > 0
                late[:, :P] = False
                for h in range(g * per, (g + 1) * per):
                    x = (s["q"][b, :, h].double() @ k.T / D ** 0.5).masked_fill(late, -math.inf)
                    out[b, :, h] = torch.softmax(x, -1) @ v
        return {"o": out}
    rot = c["rot"]
    angle = torch.zeros(B, c["S"], 1, rot // 2, dtype=torch.complex128, device=DEV)
    for j, a in enumerate(_sections(c)):
        at = s["pos"][a].long()
        angle[:, :, 0, j] = torch.complex(s["cos"][:, j].double()[at], s["sin"][:, j].double()[at])

    def turned(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        a = x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2) if c["inter"] else \
            x[..., :rot].reshape(*x.shape[:-1], 2, rot // 2).transpose(-1, -2)
        a = torch.view_as_real(torch.view_as_complex(a.contiguous()) * angle)
        x[..., :rot] = (a if c["inter"] else a.transpose(-1, -2)).reshape(*x.shape[:-1], rot)
        return x

    kc, vc = torch.zeros(s["kc"].shape, **f8), torch.zeros(s["vc"].shape, **f8)
    k, v, size = turned(s["k"], s["kw"]), s["v"].double(), s["kc"].shape[2]
    for b, n in enumerate(lens):
        row = s["row"][b, :n].long()
        page = s["table"][b].long()[row // size] if ps else torch.full_like(row, b)
        kc[page, :, row % size], vc[page, :, row % size] = k[b, :n], v[b, :n]
    return {"q": turned(s["q"], s["qw"]), "k": kc, "v": vc}
