"""GPU parity of attn_qkv_prep_axes against the definition in float64."""
from __future__ import annotations

import pytest

import serving_ref as ref
from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


def sections(half, *share):
    out = []
    for a, n in enumerate(share):
        out += [a] * n
    return (out + [len(share) - 1] * half)[:half]


def turns(half, n):
    return [j % n for j in range(half)]


# dtype, D, rot, B, S, H, G, page size, axes of the pairs, options
CASES = [
    ("bf16", 128, 128, 2, 5, 4, 2, 16, sections(64, 16, 24, 24), {}),
    ("bf16", 128, 128, 1, 1, 32, 8, 64, sections(64, 16, 24, 24), {}),
    ("f16", 128, 128, 3, 7, 6, 2, 16, turns(64, 3), dict(inter=True)),
    ("bf16", 64, 64, 2, 9, 4, 4, 0, sections(32, 16, 16), {}),
    ("f32", 64, 64, 2, 9, 4, 4, 0, sections(32, 16, 16), {}),
    ("f32", 64, 32, 2, 9, 3, 1, 5, turns(16, 2), dict(inter=True)),
    ("f16", 64, 64, 2, 11, 4, 2, 24, sections(32, 3, 10, 19), {}),            # borders inside a thread's pairs
    ("bf16", 256, 128, 2, 3, 4, 2, 16, turns(64, 4), {}),
    ("f32", 256, 256, 1, 4, 2, 2, 16, turns(128, 4), {}),
    ("bf16", 80, 80, 2, 5, 4, 2, 16, sections(40, 10, 15, 15), {}),           # rows a warp
    ("f32", 6, 6, 2, 5, 4, 2, 16, [2, 0, 1], dict(inter=True)),
    ("bf16", 128, 128, 2, 5, 4, 2, 16, sections(64, 16, 24, 24), dict(odd=3)),
    ("bf16", 128, 128, 2, 6, 4, 2, 16, turns(64, 3), dict(i8="channel")),
    ("f16", 64, 64, 2, 6, 4, 2, 0, sections(32, 8, 12, 12), dict(i8="tensor", inter=True)),
    ("bf16", 128, 128, 2, 5, 4, 2, 16, [0] * 64, {}),                         # one axis: one position a token
    ("bf16", 128, 128, 2, 5, 4, 2, 16, [3] * 64, {}),                         # ... and the last of four
    ("f16", 128, 96, 40, 50, 8, 2, 16, sections(48, 16, 16, 16), dict(nhd=True)),
    ("bf16", 128, 128, 2, 5, 4, 2, 16, sections(64, 16, 24, 24), dict(norm=False)),
    ("bf16", 128, 128, 2, 5, 4, 2, 16, sections(64, 16, 24, 24), dict(plain=True)),   # no weights, no positions
]


def definition(x, w, cos, sin, pos, axes, *, eps, norm, inter):
    """x [B, S, N, D], pos [A, B, S] -> the step in float64 and the bound of a float32 evaluation (serving_ref.prep)."""
    half = len(axes)
    c = torch.stack([cos[pos[a], j] for j, a in enumerate(axes)], -1)   # [B, S, half]
    s = torch.stack([sin[pos[a], j] for j, a in enumerate(axes)], -1)
    B, S = pos.shape[1:]
    # each token's own angles as rows of tables that serving_ref.prep reads at row b S + i
    at = torch.arange(B * S).view(B, S)
    return ref.prep(x, w, c.reshape(B * S, half), s.reshape(B * S, half), at, eps=eps, norm=norm, rot=2 * half,
                    inter=inter)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_axes(i):
    dt, D, rot, B, S, H, G, ps, axes, opt = CASES[i]
    T, g = DT[dt], torch.Generator()
    g.manual_seed(700 + i)
    odd, nhd, inter, norm = opt.get("odd", 0), opt.get("nhd", False), opt.get("inter", False), opt.get("norm", True)
    flat = (2 * torch.randn(B * S * (H + 2 * G) * D + odd, generator=g)).to(T)
    qkv = flat[odd:].view(B, S, H + 2 * G, D)
    w = [None, None] if opt.get("plain") or not norm else \
        [(1 + 0.2 * torch.randn(D, generator=g)).to(T) for _ in range(2)]
    cap, top = S + 20, S + 31
    ang = torch.arange(top, dtype=torch.float64)[:, None] * 100.0 ** -torch.linspace(0, 1, rot // 2, dtype=torch.float64)
    cos, sin = ang.cos().float(), ang.sin().float()
    pos = torch.randint(0, top, (4, B, S), generator=g).to(torch.int32)
    pos[0, 0, 0], pos[1, -1, -1] = -5, 10 ** 6   # clamped to the tables
    row = torch.stack([torch.randperm(cap, generator=g)[:S] for _ in range(B)]).to(torch.int32)
    if S > 2:
        row[0, 1], row[-1, 2] = -1, cap + 100    # tokens that write nothing
    width = -(-cap // ps) if ps else 1
    n = B * width + 2 if ps else B
    table = torch.randperm(n, generator=g)[:B * width].view(B, width).to(torch.int32)
    shape = ((n, ps, G, D) if nhd else (n, G, ps, D)) if ps else (B, G, cap, D)
    kc, vc = (torch.randint(-9, 9, shape, generator=g).to(torch.int8 if opt.get("i8") else T) for _ in range(2))
    scales = [torch.rand(G * D if opt["i8"] == "channel" else 1, generator=g) * 0.02 + 0.02 for _ in range(2)] \
        if opt.get("i8") else None
    if opt.get("plain"):
        pos = torch.arange(S, dtype=torch.int32).expand(4, B, S)
        row = torch.arange(S, dtype=torch.int32).expand(B, S)
    at = pos.long().clamp(0, top - 1)
    kw = dict(eps=1e-5, norm=norm, inter=inter)
    q, tq = definition(qkv[:, :, :H], w[0], cos, sin, at, axes, **kw)
    k, tk = definition(qkv[:, :, H:H + G], w[1], cos, sin, at, axes, **kw)
    v = qkv[:, :, H + G:].double()
    dk, dv, dqkv = kc.cuda(), vc.cuda(), flat.cuda()[odd:].view(qkv.shape)
    extra = dict(k_scale=scales[0].cuda(), v_scale=scales[1].cuda()) if scales else {}
    out = attn.qkv_prep(dqkv[:, :, :H], dqkv[:, :, H:H + G], dqkv[:, :, H + G:], dk, dv, table.cuda() if ps else None,
                        q_weight=None if w[0] is None else w[0].cuda(), k_weight=None if w[1] is None else w[1].cuda(),
                        cos=cos.cuda(), sin=sin.cuda(), positions=None if opt.get("plain") else pos.cuda(),
                        rows=None if opt.get("plain") else row.cuda(), axes=axes, eps=1e-5, norm=norm,
                        interleaved=inter, page_layout="nhd" if nhd else "hnd", **extra)
    ref.check(out, q, tq * 1.01 + ref.HALF[T] * q.abs() + 2.0 ** -25, "q")
    want_k, want_v = kc.double(), vc.double()
    tol_k, tol_v = torch.zeros_like(want_k), torch.zeros_like(want_v)
    for b in range(B):
        for t in range(S):
            r = int(row[b, t])
            if not 0 <= r < (width * ps if ps else cap):
                continue
            page, x = (int(table[b, r // ps]), r % ps) if ps else (b, r)
            for want, tol, src, e, s in ((want_k, tol_k, k, tk, 0), (want_v, tol_v, v, None, 1)):
                sel = (lambda y: y[page, x]) if nhd else (lambda y: y[page, :, x])
                y, err = src[b, t], 0 if e is None else e[b, t]
                if scales:
                    f = scales[s].double()
                    f = f.view(G, -1) if f.numel() > 1 else f
                    y, err = y / f, err / f
                    sel(want)[:], sel(tol)[:] = y.clamp(-128, 127), 0.5 + err + y.abs() * 2.0 ** -23
                else:
                    sel(want)[:] = y
                    sel(tol)[:] = 0 if e is None else err * 1.01 + ref.HALF[T] * y.abs() + 2.0 ** -25
    ref.check(dk, want_k, tol_k, "k cache")
    ref.check(dv, want_v, tol_v, "v cache")


def test_equal_positions_are_the_step_with_one_position():
    """A token with one position on every axis (text): the bits of attn_qkv_prep."""
    B, S, H, G, D = 2, 40, 8, 2, 128
    qkv = torch.randn(B, S, H + 2 * G, D, device="cuda").to(torch.bfloat16)
    cos, sin = (torch.randn(64, 64, device="cuda") for _ in range(2))
    pos = torch.randint(0, 64, (B, S), device="cuda").to(torch.int32)
    got = []
    for kw in (dict(positions=pos), dict(positions=pos.expand(3, B, S), axes=sections(64, 16, 24, 24)),
               dict(positions=pos.expand(3, B, S), axes=turns(64, 3))):
        kc, vc = (torch.zeros(B, G, S, D, dtype=qkv.dtype, device="cuda") for _ in range(2))
        out = attn.qkv_prep(qkv[:, :, :H], qkv[:, :, H:H + G], qkv[:, :, H + G:], kc, vc, cos=cos, sin=sin, **kw)
        got.append((out, kc, vc))
    for o in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, got[0]))


def test_refusals():
    B, S, H, G, D = 1, 2, 2, 1, 64
    q, k = torch.zeros(B, S, H, D, device="cuda"), torch.zeros(B, S, G, D, device="cuda")
    kc, vc = torch.zeros(B, G, 4, D, device="cuda"), torch.zeros(B, G, 4, D, device="cuda")
    t = torch.ones(9, 32, device="cuda")
    pos = torch.zeros(3, B, S, dtype=torch.int32, device="cuda")
    good = dict(cos=t, sin=t, axes=[0, 1, 2, 2] * 8, positions=pos)
    attn.qkv_prep(q, k, k, kc, vc, **good)
    for bad in (dict(axes=[0] * 31), dict(axes=[0, 4] * 16), dict(axes=[-1, 0] * 16), dict(positions=pos[:2]),
                dict(positions=pos[0]), dict(positions=pos.long()), dict(cos=None, sin=None),
                dict(positions=torch.zeros(3, B, 2 * S, dtype=torch.int32, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            attn.qkv_prep(q, k, k, kc, vc, **dict(good, **bad))
