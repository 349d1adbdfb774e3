"""Cases of the serving operators around a paged key/value cache, with their plain forms.

Three operators that one attention layer of a served model calls in turn:

* ``prep``    per-head RMS norm of Q and K, rotary position rotation, and the write of K and V
              into the cache (``attn_qkv_prep``);
* ``window``  prompt attention with a sliding window in which the first tokens (of the cache, or
              of the row's own document) stay visible (``attn_fwd_window``);
* ``paged``   attention of one new token a sequence over a paged cache, plain, windowed with first
              tokens, or quantised to int8 (``attn_decode_paged``).

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
    paged = dict(op="paged", window=-1, first=0, nhd=False)
    window = dict(op="window", docs=False, min_len=0, bshd=False)
    return [
        # one chat sequence, a short cache: a call's latency
        dict(paged, name="paged_one_short", dtype="bf16", B=1, H=32, G=8, D=128, ps=16, min_len=700, max_len=700),
        # a full serving batch with caches of very different lengths
        dict(paged, name="paged_batch64", dtype="bf16", B=64, H=32, G=8, D=128, ps=64, min_len=512, max_len=8192),
        # two very long contexts: few rows, the length must be split
        dict(paged, name="paged_two_long", dtype="f16", B=2, H=32, G=8, D=128, ps=32, min_len=100001, max_len=131072,
             nhd=True),
        # streaming chat: window plus first tokens, freed pages in between, an idle slot (length 0)
        dict(paged, name="paged_stream", dtype="bf16", B=33, H=12, G=4, D=64, ps=16, min_len=0, max_len=30011,
             window=4000, first=4, nhd=True),
        # the serving batch with an int8 cache, a scale per kv head and channel
        dict(paged, name="paged_batch64_int8", dtype="bf16", kv="i8", B=64, H=32, G=8, D=128, ps=64, min_len=512,
             max_len=8192),
        # a long prompt through a windowed layer
        dict(window, name="window_prompt", dtype="bf16", B=1, H=32, G=8, D=128, q_len=8192, k_len=8192, window=1023,
             first=4),
        # a chunk of a prompt against what is cached already
        dict(window, name="window_chunk", dtype="f16", B=2, H=16, G=2, D=128, q_len=391, k_len=16384, window=4095,
             first=64, min_len=9000),
        # packed documents, each with its own first tokens
        dict(window, name="window_docs", dtype="bf16", B=4, H=12, G=4, D=64, q_len=1024, k_len=1024, window=127,
             first=8, docs=True, bshd=True),
        # a small float32 model
        dict(window, name="window_small_f32", dtype="f32", B=1, H=2, G=2, D=32, q_len=300, k_len=300, window=63,
             first=2, bshd=True),
        # the step of a serving batch: one token a sequence, into a paged cache
        dict(op="prep", name="prep_step", dtype="bf16", B=64, S=1, H=32, G=8, D=128, rot=128, inter=False, ps=64,
             cap=256, min_len=1),
        # two long prompts into a paged cache
        dict(op="prep", name="prep_prompt", dtype="bf16", B=2, S=8192, H=32, G=8, D=128, rot=128, inter=False, ps=64,
             cap=8192, min_len=8192),
        # ragged prompts, a partial interleaved rotation, a contiguous cache, float32
        dict(op="prep", name="prep_ragged_f32", dtype="f32", B=5, S=777, H=12, G=4, D=64, rot=32, inter=True, ps=0,
             cap=1024, min_len=300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "window", "window", "prep"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while True:
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4, 8])
        if op == "paged":
            c = dict(op=op, dtype=dtype, B=_log(rng, 1, 96), H=H, G=G, D=rng.choice([64, 128, 128, 256]),
                     ps=rng.choice([8, 16, 24, 32, 64, 128]), max_len=_log(rng, 40, 131072), window=-1, first=0,
                     nhd=rng.random() < 0.5)
            c["min_len"] = int(c["max_len"] * rng.random())
            if rng.random() < 0.4:
                c["window"], c["first"] = _log(rng, 16, 8192), _log(rng, 1, 128)
            if dtype != "f32" and rng.random() < 0.25:
                c["kv"] = "i8"
            if work(c)["bytes"] <= 1.1e9 and c["B"] * c["max_len"] <= 2 ** 20:
                return c
        elif op == "window":
            q_len = _log(rng, 16, 8192)
            c = dict(op=op, dtype=dtype, B=_log(rng, 1, 8), H=H, G=G, D=rng.choice([64, 128]), q_len=q_len,
                     k_len=q_len if rng.random() < 0.6 else q_len + _log(rng, 1, 16384), window=_log(rng, 16, 4096),
                     first=_log(rng, 1, 128), docs=False, min_len=0, bshd=rng.random() < 0.5)
            if c["k_len"] > q_len:
                c["min_len"] = rng.randint(q_len, c["k_len"])
            elif rng.random() < 0.4:
                c["docs"] = True
            if dtype == "f32":
                c["D"] = rng.choice([32, 64, 128])
            pairs = c["B"] * H * q_len * c["k_len"]
            if pairs <= 2 ** 31 and work(c)["flops"] <= (1.2e11 if dtype != "f32" else 1e10):
                return c
        else:
            D = rng.choice([64, 128, 256])
            c = dict(op=op, dtype=dtype, B=_log(rng, 1, 96), S=1 if rng.random() < 0.4 else _log(rng, 2, 8192), H=H,
                     G=G, D=D, rot=rng.choice([D, D, D // 2, D // 4]), inter=rng.random() < 0.3,
                     ps=rng.choice([0, 16, 24, 64]))
            c["cap"] = c["S"] + rng.randint(0, 256)
            c["min_len"] = rng.randint(1, c["S"])
            if work(c)["bytes"] <= 4e8 and c["B"] * c["cap"] * G * D <= 2 ** 25:
                return c


def _lens(c):
    """Valid keys (paged, window) or real tokens (prep) of each batch entry."""
    r = random.Random(c["B"] * 7919 + c["min_len"])
    hi = {"paged": c.get("max_len"), "window": c.get("k_len"), "prep": c.get("S")}[c["op"]]
    lo = c["min_len"] if c["op"] != "window" or c["min_len"] else hi
    got = [r.randint(lo, hi) for _ in range(c["B"])]
    got[0], got[-1] = lo, hi   # both ends occur
    return got


def _segs(c):
    """First key of each row's document, int64 [B, q_len]: documents of 64 to 512 tokens."""
    r = random.Random(c["q_len"])
    cuts = [(b, r.randint(64, 512)) for b in range(c["B"]) for _ in range(c["q_len"] // 64 + 1)]
    n = torch.tensor([x for _, x in cuts]).view(c["B"], -1).cumsum(1)
    at = torch.arange(c["q_len"]).expand(c["B"], -1).contiguous()
    i = torch.searchsorted(n, at, right=True)
    return torch.cat([torch.zeros_like(n[:, :1]), n], 1).gather(1, i)


def _es(c):
    return 4 if c["dtype"] == "f32" else 2


def work(c):
    B, H, G, D, es = c["B"], c["H"], c["G"], c["D"], _es(c)
    lens = _lens(c)
    if c["op"] == "paged":
        hidden = [max(0, n - 1 - c["window"] - c["first"]) if c["window"] >= 0 else 0 for n in lens]
        keys = sum(lens) - sum(hidden)
        kv = 1 if c.get("kv") == "i8" else es
        rows = sum(-(-n // c["ps"]) for n in lens)
        return {"bytes": 2 * keys * G * D * kv + 2 * B * H * D * es + 4 * rows, "flops": 4 * keys * H * D}
    if c["op"] == "window":
        i = torch.arange(c["q_len"]).expand(B, -1)
        n = torch.tensor(lens)[:, None]
        diag = i + n - c["q_len"]
        seg = _segs(c) if c["docs"] else torch.zeros_like(diag)
        hi = torch.minimum(diag + 1, n)
        near = torch.maximum(diag - c["window"], seg)
        end = torch.minimum(seg + c["first"], hi)
        pairs = ((hi - torch.maximum(near, end)).clamp(min=0) + (end - seg).clamp(min=0)).sum().item()
        span = int((n.sum() if c["docs"] or c["window"] + c["first"] >= c["k_len"] else
                    (n - (n - c["q_len"] - c["window"] - c["first"]).clamp(min=0)).sum()).item())
        return {"bytes": 2 * B * c["q_len"] * H * D * es + 2 * span * G * D * es, "flops": 4 * pairs * H * D}
    tokens, real = B * c["S"], sum(lens)
    values = 2 * tokens * H * D + 4 * real * G * D + 2 * D
    return {"bytes": values * es + 2 * min(tokens, c["cap"]) * c["rot"] + 8 * tokens,
            "flops": (tokens * H + real * G) * (4 * D + 3 * c["rot"])}


# ---- inputs --------------------------------------------------------------------------------------


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _pool(g, shape, c, dtype):
    if c.get("kv") == "i8":
        return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _tables(g, counts, width):
    """Page tables: the pages of a pool in random order, -1 where an entry holds no page.
    counts: for each entry, a list of the table columns that have a page."""
    total = sum(len(cols) for cols in counts)
    perm = torch.randperm(max(total, 1), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(counts), max(width, 1)), -1, dtype=torch.int32, device=DEV)
    rows = torch.tensor([b for b, cols in enumerate(counts) for _ in cols], dtype=torch.int64, device=DEV)
    cols = torch.tensor([x for cols in counts for x in cols], dtype=torch.int64, device=DEV)
    table[rows, cols] = perm[:total]
    return table, max(total, 1)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, H, G, D, dt = c["B"], c["H"], c["G"], c["D"], DTYPES[c["dtype"]]
    lens = _lens(c)
    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if c["op"] == "paged":
        ps = c["ps"]
        live = lambda n, j: c["window"] < 0 or j * ps < c["first"] or (j + 1) * ps > n - 1 - c["window"]  # noqa: E731
        counts = [[j for j in range(-(-n // ps)) if live(n, j)] for n in lens]
        s["table"], n_pages = _tables(g, counts, -(-c["max_len"] // ps))
        shape = (n_pages, ps, G, D) if c["nhd"] else (n_pages, G, ps, D)
        s["k"], s["v"] = _pool(g, shape, c, dt), _pool(g, shape, c, dt)
        s["q"] = _normal(g, B, 1, H, D, dtype=dt)
        if c.get("kv") == "i8":
            s["ks"], s["vs"] = (torch.rand(G * D, generator=g, device=DEV) * 0.015 + 0.005 for _ in range(2))
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "window":
        hs = lambda n, h: (B, n, h, D) if c["bshd"] else (B, h, n, D)  # noqa: E731
        s["q"] = _normal(g, *hs(c["q_len"], H), dtype=dt)
        s["k"], s["v"] = (_normal(g, *hs(c["k_len"], G), dtype=dt) for _ in range(2))
        s["seg"] = _segs(c).to(torch.int32).to(DEV) if c["docs"] else None
        s["out"] = torch.empty_like(s["q"])
    else:
        S, cap, ps = c["S"], c["cap"], c["ps"]
        qkv = _normal(g, B, S, H + 2 * G, D, dtype=dt, scale=1.5)   # a packed projection, used in place
        s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + G], qkv[:, :, H + G:]
        s["qw"], s["kw"] = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt) for _ in range(2))
        i = torch.arange(S, device=DEV)[None]
        n = s["lens"][:, None]
        past = torch.randint(0, 1 << 30, (B, 1), generator=g, device=DEV) % (cap - n + 1)
        s["pos"] = torch.where(i < n, past + i, 0).to(torch.int32)
        s["row"] = torch.where(i < n, past + i, -1).to(torch.int32)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        ang = torch.arange(cap, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        width = -(-cap // ps) if ps else 1
        s["table"], n_pages = _tables(g, [list(range(width))] * B, width)
        if not ps:
            s["table"] = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
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
    if c["op"] == "prep":
        s["pages"] = attn.make_pages(c["ps"], s["kc"].shape[0], s["table"].data_ptr(), s["table"].stride(0)) \
            if c["ps"] else None
        s["plan"] = attn.make_prep(dict(
            batch=B, seq_len=c["S"], heads=H, kv_heads=G, head_dim=D, rot_dim=c["rot"], dtype=c["dtype"],
            interleaved=c["inter"], norm=True, eps=1e-6, max_pos=c["cap"], cache_rows=c["cap"],
            q_layout=strides(s["q"], 1, 2), k_layout=strides(s["k"], 1, 2), v_layout=strides(s["v"], 1, 2),
            q_out_layout=strides(s["out"], 1, 2), k_out_layout=strides(s["kc"], 2, 1),
            v_out_layout=strides(s["vc"], 2, 1)))
        return
    d = dict(batch=B, heads=H, kv_heads=G, head_dim=D, dtype=c["dtype"], causal=True, causal_align="klens",
             window_left=c["window"], masked_rows="zero")
    if c["op"] == "paged":
        row, head = (1, 2) if c["nhd"] else (2, 1)
        d.update(q_len=1, k_len=c["max_len"], q_layout=strides(s["q"], 1, 2), o_layout=strides(s["out"], 1, 2),
                 k_layout=strides(s["k"], row, head), v_layout=strides(s["v"], row, head))
        if c.get("kv") == "i8":
            d.update(kv_dtype="i8", kv_scale="channel", k_scale_ptr=s["ks"].data_ptr(), v_scale_ptr=s["vs"].data_ptr())
        s["pages"] = attn.make_pages(c["ps"], s["k"].shape[0], s["table"].data_ptr(), s["table"].stride(0))
        s["plan"] = attn.make_problem(d)
        size = attn.attn_decode_paged_workspace_size(s["plan"], s["pages"], c["first"])
    else:
        row, head = (1, 2) if c["bshd"] else (2, 1)
        d.update(q_len=c["q_len"], k_len=c["k_len"], q_layout=strides(s["q"], row, head),
                 o_layout=strides(s["out"], row, head), k_layout=strides(s["k"], row, head),
                 v_layout=strides(s["v"], row, head))
        s["plan"] = attn.make_problem(d)
        size = attn.attn_fwd_window_workspace_size(s["plan"], c["first"])
    s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)


def _own(s):
    c, attn, st = s["case"], s["attn"], torch.cuda.current_stream().cuda_stream
    ptr = torch.Tensor.data_ptr
    if c["op"] == "paged":
        rc = attn.attn_decode_paged(s["plan"], s["pages"], c["first"], ptr(s["q"]), ptr(s["k"]), ptr(s["v"]),
                                    ptr(s["out"]), None, ptr(s["lens"]), None, ptr(s["ws"]), s["ws"].numel(), st)
    elif c["op"] == "window":
        rc = attn.attn_fwd_window(s["plan"], c["first"], ptr(s["q"]), ptr(s["k"]), ptr(s["v"]), ptr(s["out"]), None,
                                  ptr(s["seg"]) if s["seg"] is not None else None, ptr(s["lens"]), None,
                                  ptr(s["ws"]), s["ws"].numel(), st)
    else:
        rc = attn.attn_qkv_prep(s["plan"], s["pages"], ptr(s["q"]), ptr(s["k"]), ptr(s["v"]), ptr(s["qw"]),
                                ptr(s["kw"]), ptr(s["cos"]), ptr(s["sin"]), ptr(s["pos"]), ptr(s["row"]),
                                ptr(s["out"]), ptr(s["kc"]), ptr(s["vc"]), st)
    if rc:
        raise attn.AttnError(rc, c["op"])
    return {"q": s["out"], "k": s["kc"], "v": s["vc"]} if c["op"] == "prep" else {"o": s["out"]}


# ---- the plain forms -----------------------------------------------------------------------------


def _softmax_pv(x, vis, v):
    """Rows of scores x (hidden ones masked by vis) against v; a row with nothing visible gives 0."""
    x = x.masked_fill(~vis, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    n = p.sum(-1, keepdim=True)
    return torch.where(n == 0, 0.0, torch.matmul(p, v) / n)


def _paged(s):
    c = s["case"]
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    at = s["table"].clamp(min=0).long()

    def rows(pool):   # [B, G, keys, D] in float32
        x = pool[at]
        return (x.permute(0, 3, 1, 2, 4) if c["nhd"] else x.permute(0, 2, 1, 3, 4)).reshape(B, G, -1, D).float()

    k, v = rows(s["k"]), rows(s["v"])
    if "ks" in s:
        k, v = k * s["ks"].view(G, 1, D), v * s["vs"].view(G, 1, D)
    q = s["q"].float().view(B, G, H // G, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    key = torch.arange(k.shape[2], device=DEV)
    n = s["lens"].view(B, 1, 1, 1)
    vis = key < n
    if c["window"] >= 0:
        vis = vis & ((key >= n - 1 - c["window"]) | (key < c["first"]))
    return {"o": _softmax_pv(x, vis, v).view(B, 1, H, D).to(s["q"].dtype)}


def _window(s):
    c = s["case"]
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    heads = (lambda t: t.transpose(1, 2)) if c["bshd"] else (lambda t: t)
    q = heads(s["q"]).float().reshape(B, G, H // G, c["q_len"], D)
    k, v = heads(s["k"]).float().unsqueeze(2), heads(s["v"]).float().unsqueeze(2)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    n = s["lens"].view(B, 1, 1)
    diag = torch.arange(c["q_len"], device=DEV).view(1, -1, 1) + n - c["q_len"]
    key = torch.arange(c["k_len"], device=DEV)
    start = s["seg"].unsqueeze(-1) if s["seg"] is not None else torch.zeros_like(diag)
    vis = (key < n) & (key <= diag) & (key >= start) & ((key >= diag - c["window"]) | (key < start + c["first"]))
    o = _softmax_pv(x, vis.view(B, 1, 1, c["q_len"], c["k_len"]), v).view(B, H, c["q_len"], D)
    return {"o": heads(o).to(s["q"].dtype).contiguous()}


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


def _prep(s):
    c = s["case"]
    pos = s["pos"].long()
    cos, sin = s["cos"][pos].unsqueeze(2), s["sin"][pos].unsqueeze(2)
    dt = s["out"].dtype
    q = _rotated(s["q"], s["qw"], cos, sin, c).to(dt)
    k = _rotated(s["k"], s["kw"], cos, sin, c).to(dt)
    real = s["row"] >= 0
    b, i = torch.nonzero(real, as_tuple=True)
    row = s["row"][b, i].long()
    ps = s["kc"].shape[2]
    page = s["table"][b, row // ps].long()
    s["kc"].transpose(1, 2)[page, row % ps] = k[b, i]
    s["vc"].transpose(1, 2)[page, row % ps] = s["v"][b, i]
    return {"q": q, "k": s["kc"], "v": s["vc"]}


def run(s):
    if own:
        return _own(s)
    return {"paged": _paged, "window": _window, "prep": _prep}[s["case"]["op"]](s)


# ---- 64 bits, from the definitions -----------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    per = H // G
    lens = _lens(c)
    f8 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "paged":
        out = torch.zeros(B, 1, H, D, **f8)
        for b, n in enumerate(lens):
            keys = [j for j in range(n) if c["window"] < 0 or j < c["first"] or n - 1 - j <= c["window"]]
            if not keys:
                continue
            keys = torch.tensor(keys, device=DEV)
            page, r = s["table"][b].long()[keys // c["ps"]], keys % c["ps"]
            for g in range(G):
                k, v = ((p[page, r, g] if c["nhd"] else p[page, g, r]).double() for p in (s["k"], s["v"]))
                if c.get("kv") == "i8":
                    k, v = k * s["ks"][g * D:(g + 1) * D].double(), v * s["vs"][g * D:(g + 1) * D].double()
                w = torch.softmax(s["q"][b, 0, g * per:(g + 1) * per].double() @ k.T / D ** 0.5, -1)
                out[b, 0, g * per:(g + 1) * per] = w @ v
        return {"o": out}
    if c["op"] == "window":
        q, k, v = (t.transpose(1, 2) if c["bshd"] else t for t in (s["q"], s["k"], s["v"]))
        out = torch.zeros(B, H, c["q_len"], D, **f8)
        step = 256
        for b, n in enumerate(lens):
            for i0 in range(0, c["q_len"], step):
                i = torch.arange(i0, min(i0 + step, c["q_len"]), device=DEV)
                last = i + n - c["q_len"]                                    # a row's own key
                start = s["seg"][b, i].long() if c["docs"] else torch.zeros_like(i)
                spans = torch.zeros(c["k_len"] + 1, dtype=torch.bool, device=DEV)
                spans[max(0, int(last[0]) - c["window"]):int(last[-1]) + 1] = True
                for f in start.unique().tolist():
                    spans[f:f + c["first"]] = True
                keys = spans[:c["k_len"]].nonzero()[:, 0]
                keys = keys[keys < n]
                d = last[:, None] - keys
                from_start = keys - start[:, None]
                hide = (d < 0) | (from_start < 0) | ((d > c["window"]) & (from_start >= c["first"]))
                kk, vv = k[b][:, keys].double(), v[b][:, keys].double()
                for h in range(H):
                    x = (q[b, h, i].double() @ kk[h // per].T / D ** 0.5).masked_fill(hide, -math.inf)
                    out[b, h, i] = torch.nan_to_num(torch.softmax(x, -1)) @ vv[h // per]
        return {"o": (out.transpose(1, 2) if c["bshd"] else out).contiguous()}
    rot = c["rot"]
    pos = s["pos"].long()
    angle = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, :, None]

    def turned(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        a = x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2) if c["inter"] else \
            x[..., :rot].reshape(*x.shape[:-1], 2, rot // 2).transpose(-1, -2)
        a = torch.view_as_real(torch.view_as_complex(a.contiguous()) * angle)
        x[..., :rot] = (a if c["inter"] else a.transpose(-1, -2)).reshape(*x.shape[:-1], rot)
        return x

    kc, vc = torch.zeros(s["kc"].shape, **f8), torch.zeros(s["vc"].shape, **f8)
    k, v, ps = turned(s["k"], s["kw"]), s["v"].double(), s["kc"].shape[2]
    for b, n in enumerate(lens):
        row = s["row"][b, :n].long()
        page = s["table"][b].long()[row // ps]
        kc[page, :, row % ps], vc[page, :, row % ps] = k[b, :n], v[b, :n]
    return {"q": turned(s["q"], s["qw"]), "k": kc, "v": vc}
