"""Additive masks with values down to float32's lowest, in windows with first keys
and in paged decode: they hide nothing by themselves.  A row whose visible keys
all carry the lowest value has the mean of their V (its scores are absorbed), a
key beside a higher value has no weight, and only -inf takes a key out."""
from __future__ import annotations

import pytest

import serving_bounds as sb
from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LOW = sb.LOW


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


@pytest.mark.parametrize("dt,D,H,G,Sq,Sk,w,first,opt", [
    ("bf16", 128, 4, 2, 300, 700, 90, 5, {}),
    ("f16", 64, 4, 2, 300, 300, 90, 40, dict(sink=True)),
    ("bf16", 64, 2, 2, 60, 3000, 900, 3, {}),                  # parts that meet in a cluster
    ("f16", 128, 2, 1, 70, 1500, 800, 7, dict(splits=4)),      # and in the workspace
    ("bf16", 128, 2, 2, 200, 400, 90, 5, dict(softcap=20.0)),
    ("f16", 96, 2, 1, 60, 200, 50, 4, {}),
    ("f32", 64, 4, 2, 200, 500, 90, 5, {}),
    ("f32", 128, 2, 1, 40, 900, 500, 5, dict(splits=3, sink=True)),
    ("f32", 32, 2, 2, 90, 90, 20, 2, dict(softcap=5.0)),
    ("f32", 48, 2, 2, 50, 90, 20, 2, {}),
])
def test_window_masks(dt, D, H, G, Sq, Sk, w, first, opt):
    g = gen(3 + D + Sq)
    q, k, v = (randn(g, 1, h, n, D, dt=DT[dt]) for h, n in ((H, Sq), (G, Sk), (G, Sk)))
    mask = sb.mask_kinds(g, 1, 1, Sq, Sk)
    sink = randn(g, H) if opt.get("sink") else None
    i, j = torch.arange(Sq, device="cuda")[:, None] + Sk - Sq, torch.arange(Sk, device="cuda")[None]
    vis = ((j <= i) & ((j >= i - w) | (j < first)))[None]
    o, lse, tol, tol_l = sb.attention(q, k, v, vis, p="single", mask=mask, sink=sink, softcap=opt.get("softcap", 0.0))
    got, got_l = attn.fwd(q, k, v, layout="bhsd", causal=True, window_left=w, first_keys=first, mask=mask,
                          head_sink=sink, softcap=opt.get("softcap", 0.0), key_splits=opt.get("splits", 0),
                          masked_rows="zero", return_lse=True)
    sb.check(got, o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")
    assert sink is not None or (lse == LOW).any()   # rows that are the mean of their keys are among them


@pytest.mark.parametrize("dt,D,H,G,B,rows,opt", [
    ("bf16", 128, 8, 2, 2, 500, {}),                   # clusters
    ("f16", 64, 8, 8, 60, 100, dict(sink=True)),       # whole units
    ("f16", 64, 8, 8, 58, 1800, {}),                   # shares
    ("bf16", 128, 16, 8, 58, 900, dict(softcap=9.0)),
    ("bf16", 128, 8, 2, 2, 500, dict(i8=True)),
    ("f16", 128, 16, 8, 58, 1700, dict(i8=True)),
    ("f32", 64, 8, 2, 2, 500, {}),
    ("f32", 128, 16, 8, 60, 60, {}),
    ("f32", 64, 16, 8, 58, 900, dict(sink=True)),
    ("f16", 80, 4, 2, 3, 200, {}),
])
def test_paged_masks(dt, D, H, G, B, rows, opt):
    g, ps = gen(5 + D + B), 16
    i8 = opt.get("i8")
    if i8:
        k, v = (torch.randint(-128, 128, (60, G, ps, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
        sc = [torch.rand(G * D, generator=g, device="cuda") * 0.015 + 0.005 for _ in range(2)]
    else:
        k, v, sc = randn(g, 60, G, ps, D, dt=DT[dt]), randn(g, 60, G, ps, D, dt=DT[dt]), None
    q = randn(g, B, 1, H, D, dt=DT[dt])
    table = torch.randint(0, 60, (B, -(-rows // ps)), generator=g, device="cuda").to(torch.int32)
    n = torch.randint(rows // 2, rows + 1, (B,), generator=g, device="cuda").to(torch.int32)
    mask = sb.mask_kinds(g, B, H, 1, rows)
    sink = randn(g, H) if opt.get("sink") else None
    vis = (torch.arange(rows, device="cuda")[None] < n[:, None])[:, None]
    o, lse, tol, tol_l = sb.attention(q.transpose(1, 2), sb.rows_of(k, table, ps, rows), sb.rows_of(v, table, ps, rows),
                                      vis, mask=mask, sink=sink, softcap=opt.get("softcap", 0.0), kv_scales=sc,
                                      extra_score=2.0 ** -22 if i8 else 0.0)
    kw = dict(k_scale=sc[0], v_scale=sc[1]) if i8 else {}
    got, got_l = attn.decode_paged(q, k, v, table, n, mask=mask, head_sink=sink, softcap=opt.get("softcap", 0.0),
                                   max_rows=rows, masked_rows="zero", return_lse=True, **kw)
    sb.check(got.transpose(1, 2), o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")
    assert sink is not None or (lse == LOW).any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_lowest_sinks(dt):
    """A sink of the lowest value beside no key is a row of zeros with that LSE; beside keys it weighs nothing."""
    g = gen(11)
    q, pool = randn(g, 2, 1, 4, 64, dt=DT[dt]), randn(g, 8, 2, 16, 64, dt=DT[dt])
    table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
    n = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    sink = torch.full((4,), LOW, device="cuda")
    got, lse = attn.decode_paged(q, pool, pool, table, n, head_sink=sink, return_lse=True)
    plain = attn.decode_paged(q, pool, pool, table, n, masked_rows="zero")
    assert torch.equal(got, plain) and (lse[0] == LOW).all() and torch.isfinite(lse).all()
    kv = randn(g, 1, 2, 64, 64, dt=DT[dt])
    qq = randn(g, 1, 4, 64, 64, dt=DT[dt])
    kw = dict(layout="bhsd", causal=True, causal_offset=-5, window_left=20, first_keys=3)
    got, lse = attn.fwd(qq, kv, kv, head_sink=sink, return_lse=True, **kw)
    assert torch.equal(got, attn.fwd(qq, kv, kv, masked_rows="zero", **kw))
    assert (lse[:, :, :5] == LOW).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt,D,splits", [("f32", 64, 0), ("f32", 48, 5), ("bf16", 64, 6), ("f16", 96, 2), ("f16", 128, 16)])
@pytest.mark.parametrize("room", [0, 1 << 16])
def test_masked_parts_stay_in_the_workspace(dt, D, splits, room):
    """The workspace the query asks for holds masked parts and their sums (fewer parts), a larger one all parts."""
    g, guard = gen(D + splits), 1 << 12
    H, G, Sq, Sk, w, first = 2, 1, 40, 2000, 1500, 5
    q, k, v = (randn(g, 1, h, n, D, dt=DT[dt]) for h, n in ((H, Sq), (G, Sk), (G, Sk)))
    mask = sb.mask_kinds(g, 1, 1, Sq, Sk)
    out, lse = torch.empty_like(q), torch.empty(1, H, Sq, device="cuda")
    p = attn.make_problem(dict(
        batch=1, heads=H, kv_heads=G, q_len=Sq, k_len=Sk, head_dim=D, dtype=dt, causal=True, window_left=w,
        masked_rows="zero", key_splits=splits, mask_layout=(0, 0, 0, mask.stride(2)), lse_layout=lse.stride()[:2],
        **{f"{n}_layout": attn._layout4(t, 1) for n, t in (("q", q), ("k", k), ("v", v), ("o", out))}))
    size = attn.attn_fwd_window_workspace_size(p, first)
    assert size
    size += room
    ws = torch.full((size + 2 * guard,), 171, dtype=torch.uint8, device="cuda")
    assert attn.attn_fwd_window(p, first, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), mask.data_ptr(), None,
                                None, lse.data_ptr(), ws.data_ptr() + guard, size,
                                torch.cuda.current_stream().cuda_stream) == 0
    i, j = torch.arange(Sq, device="cuda")[:, None] + Sk - Sq, torch.arange(Sk, device="cuda")[None]
    vis = ((j <= i) & ((j >= i - w) | (j < first)))[None]
    o, l, tol, tol_l = sb.attention(q, k, v, vis, p="single", mask=mask)
    sb.check(out, o, tol, "O")
    sb.check(lse, l, tol_l, "LSE")
    assert (ws[:guard] == 171).all() and (ws[guard + size:] == 171).all()
