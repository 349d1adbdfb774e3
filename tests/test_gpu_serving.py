"""GPU parity of attn_fwd_window, attn_decode_paged and attn_qkv_prep against
the float64 references and bounds of serving_ref.py, at the sizes, masks,
layouts and lists where they can go wrong, and a run of the three together."""
from __future__ import annotations

import math

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


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dt)


# ---- windows with first keys -----------------------------------------------------------------------

# dtype, D, B, H, G, q_len, k_len, window, first, options
WINDOW = [
    ("bf16", 128, 1, 4, 2, 700, 700, 127, 4, {}),
    ("bf16", 128, 2, 2, 1, 513, 1500, 200, 130, dict(lens=[1500, 900])),
    ("f16", 64, 2, 6, 2, 390, 1000, 63, 1, dict(lens=[0, 1000])),          # an entry without keys
    ("f16", 128, 1, 2, 2, 1, 600, 31, 5, {}),
    ("bf16", 64, 2, 3, 1, 100, 2000, 255, 16, dict(splits=5)),             # paired heads, an odd count, parts
    ("f16", 128, 1, 2, 1, 300, 3000, 1500, 7, dict(splits=16, lens=[2222])),
    ("bf16", 64, 3, 2, 2, 600, 600, 63, 8, dict(docs=97)),
    ("f16", 128, 2, 2, 1, 515, 515, 0, 1, dict(docs=260)),                 # a window of the row's own key
    ("bf16", 128, 1, 2, 2, 400, 400, 50, 500, {}),                         # more first keys than keys
    ("bf16", 128, 1, 2, 2, 400, 400, 399, 3, {}),                          # a window that hides nothing
    ("f16", 64, 1, 2, 1, 640, 640, 129, 127, dict(mask="row", softcap=20.0)),
    ("bf16", 128, 2, 4, 2, 300, 700, 100, 3, dict(mask="bcast", zero=False)),
    ("bf16", 128, 1, 4, 4, 300, 900, 100, 129, dict(sink=True)),
    ("f16", 64, 1, 2, 1, 200, 800, 90, 4, dict(smooth=True, splits=3)),
    ("bf16", 128, 1, 2, 2, 300, 300, 40, 6, dict(scale=-0.07)),
    ("f16", 256, 1, 2, 1, 300, 900, 150, 9, {}),
    ("bf16", 256, 2, 2, 2, 130, 500, 60, 140, dict(docs=0, lens=[500, 333])),
    ("bf16", 256, 1, 2, 1, 300, 300, 40, 6, dict(docs=77)),
    ("f32", 32, 1, 2, 2, 300, 300, 63, 2, {}),
    ("f32", 128, 2, 4, 2, 130, 400, 50, 33, dict(lens=[400, 260])),
    ("f32", 64, 1, 2, 1, 70, 900, 300, 5, dict(splits=4, sink=True)),
    ("f32", 80, 1, 3, 1, 65, 65, 10, 3, dict(docs=20)),
    ("f32", 5, 1, 1, 1, 40, 64, 7, 2, dict(mask="row")),
    ("f16", 96, 1, 4, 2, 100, 150, 20, 10, {}),
    ("bf16", 128, 1, 2, 1, 200, 500, 64, 4, dict(offset=500)),             # rows whose window is behind the keys
    ("bf16", 128, 1, 2, 1, 200, 500, 64, 4, dict(offset=-120, zero=False)),  # rows in front of every key
]


def window_case(c, seed, bshd):
    dt, D, B, H, G, Sq, Sk, w, first, opt = c
    g, dt = gen(seed), DT[dt]
    q, k, v = randn(g, B, H, Sq, D, dt=dt), randn(g, B, G, Sk, D, dt=dt), randn(g, B, G, Sk, D, dt=dt)
    lens = opt.get("lens", [Sk] * B)
    seg = None
    if opt.get("docs"):
        seg = (torch.arange(Sq) // opt["docs"] * opt["docs"]).to(torch.int32).expand(B, Sq).contiguous()
    mask = None
    if opt.get("mask"):
        mask = randn(g, B, 1, 1 if opt["mask"] == "bcast" else Sq, Sk)
        mask[torch.rand(mask.shape, generator=g) < 0.3] = -math.inf
        mask[..., 7] = torch.finfo(torch.float32).min   # the type's lowest value is no -inf
        mask[0, :, -1, :] = -math.inf                   # (bcast: every row of the entry is empty)
    sink = randn(g, H) if opt.get("sink") else (torch.zeros(H) if opt.get("smooth") else None)
    vis = ref.visible(Sq, Sk, lens, offset=opt.get("offset"), window=w, first=first, seg=seg)
    dead = ~vis.any(1)   # keys no row sees: NaN where no tile of the kernels mixes them in
    want = ref.attention(q, k, v, vis, mask=mask, softcap=opt.get("softcap", 0.0), sink=sink,
                         zero=opt.get("zero", True), scale=opt.get("scale", 0.0))
    k = torch.where(dead[:, None, :, None], math.nan, k)
    v = torch.where(dead[:, None, :, None], math.nan, v)
    ten = [t.transpose(1, 2).contiguous() if bshd else t for t in (q, k, v)]
    kw = dict(layout="bshd" if bshd else "bhsd", causal=True, window_left=w, first_keys=first, return_lse=True,
              masked_rows="zero" if opt.get("zero", True) else "nan", softcap=opt.get("softcap", 0.0),
              key_splits=opt.get("splits", 0), scale=opt.get("scale", 0.0))
    if "offset" in opt:
        kw.update(causal_offset=opt["offset"])
    else:
        kw.update(causal_align="klens", k_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    kw.update(seg=None if seg is None else seg.cuda(), mask=None if mask is None else mask.cuda(),
              head_sink=sink.cuda() if opt.get("sink") else None, smooth_softmax=bool(opt.get("smooth")))
    return [t.cuda() for t in ten], kw, want


@pytest.mark.parametrize("i", range(len(WINDOW)))
@pytest.mark.parametrize("bshd", [False, True])
def test_window(i, bshd):
    (q, k, v), kw, (o, lse, tol, tol_l) = window_case(WINDOW[i], 100 + i, bshd)
    got, got_l = attn.fwd(q, k, v, **kw)
    assert attn.attn_device_status() == attn.ATTN_OK
    ref.check(got.transpose(1, 2) if bshd else got, o, tol, "O")
    ref.check(got_l, lse, tol_l, "LSE")
    again, again_l = attn.fwd(q, k, v, **kw)
    assert torch.equal(got.nan_to_num(7.0), again.nan_to_num(7.0)) and torch.equal(got_l, again_l)


def test_window_many_items_a_cta():
    """More query blocks than SMs: each CTA runs several items, with entries of no, few and all keys between."""
    c = ("bf16", 64, 5, 8, 2, 1100, 1400, 200, 3, dict(lens=[1400, 0, 1100, 7, 1250]))
    (q, k, v), kw, (o, lse, tol, tol_l) = window_case(c, 77, False)
    got, got_l = attn.fwd(q, k, v, **kw)
    ref.check(got, o, tol, "O")
    ref.check(got_l, lse, tol_l, "LSE")


def test_window_bounded_wait():
    """A copy that never lands ends in a status; the next call is right."""
    (q, k, v), kw, (o, lse, tol, tol_l) = window_case(WINDOW[0], 100, False)
    attn.attn_test_inject(attn.ATTN_INJECT_DROP_FIRST_COPY)
    attn.fwd(q, k, v, **kw)
    assert attn.attn_device_status() == attn.ATTN_ERR_DEVICE_TIMEOUT
    got, got_l = attn.fwd(q, k, v, **kw)
    assert attn.attn_device_status() == attn.ATTN_OK
    ref.check(got, o, tol, "O")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("step,every", [(32, 20), (32, 130), (4, 7), (-32, 20), (64, 33)])
def test_window_rising_scores(dt, step, every):
    """Scores that climb (or fall) by `step` every few keys: running maxima move inside tiles and between them."""
    g = gen(35)
    Sq, Sk, D = 300, 400, 64
    q, k = torch.zeros(1, 2, Sq, D, dtype=DT[dt]), torch.zeros(1, 1, Sk, D, dtype=DT[dt])
    q[..., 0] = 1
    k[0, 0, :, 0] = (torch.arange(Sk) // every * step).to(DT[dt])   # exact in every type
    v = randn(g, 1, 1, Sk, D, dt=DT[dt])
    vis = ref.visible(Sq, Sk, [Sk], window=200, first=40)
    o, lse, tol, tol_l = ref.attention(q, k, v, vis, scale=1.0)
    got, got_l = attn.fwd(q.cuda(), k.cuda(), v.cuda(), layout="bhsd", causal=True, window_left=200, first_keys=40,
                          scale=1.0, return_lse=True)
    ref.check(got, o, tol, "O")
    ref.check(got_l, lse, tol_l, "LSE")
    # and the same keys in pages
    pool = [t[0].view(1, 25, 16, D).transpose(0, 1).contiguous().cuda() for t in (k, v)]
    table = torch.arange(25, dtype=torch.int32).view(1, 25).cuda()
    vis = ref.visible(1, Sk, [Sk], window=200, first=40)
    o, lse, tol, tol_l = ref.attention(q[:, :, :1], k, v, vis, scale=1.0)
    got, got_l = attn.decode_paged(q[:, :, :1].transpose(1, 2).contiguous().cuda(), *pool, table,
                                   torch.tensor([Sk], dtype=torch.int32).cuda(), window_left=200, first_keys=40,
                                   scale=1.0, return_lse=True)
    ref.check(got.transpose(1, 2), o, tol, "paged O")
    ref.check(got_l, lse, tol_l, "paged LSE")


@pytest.mark.parametrize("dt,lead,pad", [("bf16", 8, 8), ("f16", 16, 24), ("f32", 4, 4), ("f32", 1, 1), ("bf16", 1, 3),
                                         ("bf16", 0, 8)])
def test_window_strided_views(dt, lead, pad):
    """Rows inside wider ones that start off 32, 16 or even 4 bytes; what lies between the rows of O stays."""
    g = gen(31)
    B, H, G, Sq, Sk, D = 2, 4, 2, 140, 300, 64

    def view(h, n, fill=None):
        flat = torch.full((lead + B * n * h * (D + pad),), 5.0) if fill else randn(g, lead + B * n * h * (D + pad))
        return flat.to(DT[dt]).cuda()[lead:].view(B, n, h, D + pad)[..., :D]

    q, k, v, out = view(H, Sq), view(G, Sk), view(G, Sk), view(H, Sq, True)
    attn.fwd(q, k, v, layout="bshd", causal=True, window_left=33, first_keys=5, masked_rows="zero", out=out)
    vis = ref.visible(Sq, Sk, [Sk] * B, window=33, first=5)
    o, _, tol, _ = ref.attention(*(t.cpu().transpose(1, 2) for t in (q, k, v)), vis)
    ref.check(out.transpose(1, 2), o, tol)
    rest = out.as_strided(out.shape[:3] + (pad,), out.stride(), out.storage_offset() + D)
    assert (rest[:, :-1] == 5).all()


def test_window_int8_keys_and_values():
    g = gen(33)
    H, G, Sq, Sk, D = 4, 2, 70, 200, 64
    q = randn(g, 1, H, Sq, D, dt=torch.bfloat16)
    k, v = (torch.randint(-128, 128, (1, G, Sk, D), generator=g, dtype=torch.int8) for _ in range(2))
    sc = [torch.rand(G * D, generator=g) * 0.015 + 0.005 for _ in range(2)]
    vis = ref.visible(Sq, Sk, [Sk], window=20, first=6)
    o, _, tol, _ = ref.attention(q, k, v, vis, kv_scales=sc)
    qd, kd, vd, ks, vs = (t.cuda() for t in (q, k, v, *sc))
    out = torch.empty_like(qd)
    p = attn.make_problem(dict(
        batch=1, heads=H, kv_heads=G, q_len=Sq, k_len=Sk, head_dim=D, dtype="bf16", causal=True, window_left=20,
        kv_dtype="i8", kv_scale="channel", k_scale_ptr=ks.data_ptr(), v_scale_ptr=vs.data_ptr(),
        **{f"{n}_layout": attn._layout4(t, 1) for n, t in (("q", qd), ("k", kd), ("v", vd), ("o", out))}))
    assert attn.attn_fwd_window(p, 6, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), out.data_ptr(), None, None, None,
                                None, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    ref.check(out, o, tol)


def test_window_shared_workspace_and_graphs():
    """Two captured calls that share a workspace of parts, replayed in turn, and an eager call between."""
    cases = [window_case(WINDOW[i], 50 + i, False) for i in (4, 5)]
    want = [attn.fwd(*t, **kw) for t, kw, _ in cases]
    graphs, outs = [], []
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")
    for (q, k, v), kw, _ in cases:
        out = torch.empty_like(q)
        p = attn.make_problem(dict(
            batch=q.shape[0], heads=q.shape[1], kv_heads=k.shape[1], q_len=q.shape[2], k_len=k.shape[2],
            head_dim=q.shape[3], dtype=attn._dtype_name(q), causal=True, causal_align="klens",
            window_left=kw["window_left"], masked_rows="zero", key_splits=kw["key_splits"],
            **{f"{n}_layout": attn._layout4(t, 1) for n, t in (("q", q), ("k", k), ("v", v), ("o", out))}))
        assert 0 < attn.attn_fwd_window_workspace_size(p, kw["first_keys"]) <= ws.numel()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            assert attn.attn_fwd_window(p, kw["first_keys"], q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                        None, None, kw["k_lens"].data_ptr(), None, ws.data_ptr(), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream) == 0
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g, out, (o, _) in zip(graphs, outs, want):
            out.zero_()
            ws.fill_(255)
            g.replay()
            assert torch.equal(out, o)


def test_window_without_first_keys_is_attn_fwd():
    (q, k, v), kw, _ = window_case(WINDOW[0], 3, False)
    kw = dict(kw, first_keys=0)
    a, la = attn.fwd(q, k, v, **kw)
    d = dict(batch=1, heads=4, kv_heads=2, q_len=700, k_len=700, head_dim=128, dtype="bf16", causal=True,
             causal_align="klens", window_left=127, masked_rows="zero",
             **{f"{n}_layout": attn._layout4(t, 1) for n, t in (("q", q), ("k", k), ("v", v), ("o", a))})
    p, o = attn.make_problem(d), torch.empty_like(a)
    n = attn.attn_fwd_window_workspace_size(p, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert attn.attn_fwd_window(p, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), None, None,
                                kw["k_lens"].data_ptr(), None, ws.data_ptr() if n else None, n,
                                torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(a, o)


# ---- paged caches ----------------------------------------------------------------------------------

# dtype, D, H, G, page_size, lens, options
PAGED = [
    ("bf16", 128, 8, 2, 16, [0, 1, 15, 16, 17, 900], {}),
    ("f16", 128, 8, 8, 64, [2500, 63, 64, 65], dict(nhd=True)),
    ("bf16", 64, 6, 2, 32, [700, 33, 31], {}),
    ("f16", 256, 4, 2, 16, [300, 129], dict(nhd=True)),
    ("bf16", 256, 24, 1, 64, [300, 1], {}),                                  # more heads than one CTA takes
    ("bf16", 128, 34, 2, 8, [500, 40], {}),
    ("f16", 128, 4, 4, 24, [1000, 23, 25], {}),                              # pages that end inside a tile
    ("bf16", 64, 4, 1, 1, [150, 3], dict(nhd=True)),                         # a page a token
    ("f16", 64, 5, 5, 7, [200, 8], {}),
    ("bf16", 128, 4, 2, 100, [777, 100, 101], {}),
    ("bf16", 128, 4, 2, 300, [777, 100, 301], {}),
    ("bf16", 128, 8, 2, 16, [3000, 40, 0, 130], dict(window=100, first=4)),
    ("f16", 64, 4, 2, 32, [2000, 70, 64], dict(window=255, first=130, nhd=True)),
    ("bf16", 128, 4, 2, 16, [500, 400], dict(window=0, first=1)),
    ("bf16", 128, 4, 2, 16, [500, 400], dict(window=63, first=0)),
    ("bf16", 128, 4, 2, 16, [600, 90], dict(bad=True)),                      # lists that name no page
    ("f32", 64, 4, 2, 16, [600, 90], dict(bad=True)),
    ("f16", 128, 8, 4, 16, [300, 200], dict(mask=True, softcap=30.0, zero=False)),
    ("bf16", 64, 8, 4, 16, [300, 0], dict(mask=True, sink=True)),
    ("f16", 128, 4, 4, 32, [300, 0], dict(smooth=True)),
    ("f32", 128, 8, 2, 16, [900, 1, 0, 17], {}),
    ("f32", 64, 6, 2, 24, [700, 33], dict(nhd=True, window=50, first=30)),
    ("f32", 256, 2, 1, 32, [333], dict(softcap=5.0)),
    ("f32", 80, 3, 3, 5, [100, 64], {}),
    ("f32", 128, 24, 1, 16, [400, 4], dict(mask=True)),
    ("f16", 96, 4, 2, 16, [333, 20], {}),
    ("bf16", 2, 2, 1, 16, [100], {}),
    ("bf16", 128, 8, 2, 16, [1000, 17, 0], dict(i8="channel")),
    ("f16", 128, 8, 1, 24, [1000, 47], dict(i8="tensor", nhd=True)),
    ("bf16", 64, 12, 1, 32, [600, 2], dict(i8="channel", window=99, first=3)),
    ("f16", 128, 4, 2, 64, [300, 20], dict(i8="channel", mask=True, softcap=9.0)),
    ("bf16", 128, 4, 2, 16, [300, 200], dict(i8="channel", bad=True)),
    ("f16", 256, 4, 2, 16, [300, 20], dict(i8="channel")),
    ("f32", 64, 4, 2, 16, [300, 20], dict(i8="tensor")),
    ("bf16", 128, 4, 2, 16, [600, 90], dict(slack=16)),                      # rows with a stride of their own
    ("bf16", 128, 4, 2, 16, [600, 90], dict(slack=3)),                       # and one no 16-byte load can take
    ("f32", 128, 4, 2, 16, [200, 90], dict(slack=1)),
    ("bf16", 128, 4, 2, 16, [600, 90], dict(cap=500)),                       # lengths beyond max_rows
    ("bf16", 128, 2, 2, 16, [9000], {}),
    # long lists and many units: shares that cut units, entries without keys among them
    ("bf16", 128, 8, 2, 16, [9000, 0, 4321, 1], dict(nhd=True)),
    ("f16", 64, 6, 2, 64, [6000, 4097, 17], dict(window=5000, first=200)),
    ("f32", 64, 4, 2, 16, [5000, 0, 3], dict(sink=True)),
    ("f32", 128, 6, 1, 32, [7000, 5000], {}),
    ("bf16", 128, 4, 1, 32, [9000, 8191], dict(i8="channel")),
    ("f16", 128, 20, 1, 16, [5000, 4500], dict(mask=True, zero=False)),
    ("f16", 256, 2, 1, 16, [5000, 77], dict(smooth=True)),
    ("bf16", 64, 8, 8, 16, [37 * i % 500 for i in range(70)], {}),
    ("f32", 64, 8, 8, 8, [29 * i % 200 for i in range(70)], dict(bad=True)),
    ("f16", 128, 8, 8, 16, [61 * i % 400 for i in range(65)], dict(window=50, first=3, sink=True)),
    ("bf16", 128, 2, 1, 16, [0, 0, 0], dict(sink=True)),
    ("f16", 128, 8, 8, 16, [0] * 60, dict(zero=False)),
]


def paged_case(c, seed):
    dt, D, H, G, ps, lens, opt = c
    g, dt, B = gen(seed), DT[dt], len(lens)
    nhd, w, first = opt.get("nhd", False), opt.get("window", -1), opt.get("first", 0)
    width = max(-(-max(lens) // ps), 1) + 1
    used = [[j for j in range(-(-n // ps)) if w < 0 or j * ps < first or (j + 1) * ps > n - 1 - w] for n in lens]
    n_pages = sum(map(len, used)) + 3
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, cols in enumerate(used):
        for j in cols:
            table[b, j] = int(perm[at])
            at += 1
        table[b, len(range(-(-lens[b] // ps))):] = 2 ** 31 - 1 if b % 2 else -7   # padding that must not be used
    if opt.get("bad"):
        table[0, 1], table[0, 3], table[1, :] = -1, n_pages, -2 ** 31
    cap = opt.get("cap", width * ps)
    shape = (n_pages, ps, G, D) if nhd else (n_pages, G, ps, D)
    slack = opt.get("slack", 0)
    wide = shape[:3] + (D + slack,)
    scales = None
    if opt.get("i8"):
        k, v = (torch.randint(-128, 128, wide, generator=g, dtype=torch.int8) for _ in range(2))
        scales = [torch.rand(G * D if opt["i8"] == "channel" else 1, generator=g) * 0.015 + 0.005 for _ in range(2)]
    else:
        k, v = randn(g, *wide, dt=dt), randn(g, *wide, dt=dt)
    k, v = k[..., :D], v[..., :D]
    q = randn(g, B, 1, H, D, dt=dt)
    rk, ok = ref.gather(k, table, ps, cap, nhd)
    rv, _ = ref.gather(v, table, ps, cap, nhd)
    vis = ref.visible(1, cap, [min(n, cap) for n in lens], window=w, first=first) & ok[:, None]
    mask = None
    if opt.get("mask"):
        mask = randn(g, B, H, 1, cap)
        mask[torch.rand(mask.shape, generator=g) < 0.3] = -math.inf
        mask[-1, 0] = -math.inf
    sink = randn(g, H) if opt.get("sink") else (torch.zeros(H) if opt.get("smooth") else None)
    want = ref.attention(q.transpose(1, 2), rk, rv, vis, mask=mask, softcap=opt.get("softcap", 0.0), sink=sink,
                         zero=opt.get("zero", True), kv_scales=scales, half_q=bool(scales) and dt != torch.float32)
    if not opt.get("i8"):   # rows nothing sees are never read
        seen = torch.zeros(n_pages, ps, dtype=torch.bool)
        b, r = torch.nonzero(vis[:, 0], as_tuple=True)
        seen[table[b, r // ps].long(), r % ps] = True
        hide = ~(seen[:, :, None, None] if nhd else seen[:, None, :, None])
        k, v = (torch.where(hide, math.nan, t) for t in (k, v))
        if slack:
            k, v = (torch.nn.functional.pad(t, (0, slack))[..., :D] for t in (k, v))
    if slack:
        k, v = (torch.as_strided(t.cuda(), t.shape, t.stride()) if t.cuda().stride() == t.stride()
                else _keep_strides(t, slack) for t in (k, v))
    kw = dict(page_layout="nhd" if nhd else "hnd", masked_rows="zero" if opt.get("zero", True) else "nan",
              window_left=None if w < 0 else w, first_keys=first, softcap=opt.get("softcap", 0.0),
              mask=None if mask is None else mask.cuda(), head_sink=sink.cuda() if opt.get("sink") else None,
              smooth_softmax=bool(opt.get("smooth")), max_rows=cap)
    if scales:
        kw.update(k_scale=scales[0].cuda(), v_scale=scales[1].cuda())
    args = (q.cuda(), k.cuda() if not slack else k, v.cuda() if not slack else v, table.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda())
    return args, kw, want


def _keep_strides(t, slack):
    wide = torch.zeros(t.shape[:3] + (t.shape[3] + slack,), dtype=t.dtype, device="cuda")
    wide[..., :t.shape[3]] = t.cuda()
    return wide[..., :t.shape[3]]


@pytest.mark.parametrize("i", range(len(PAGED)))
def test_paged(i):
    args, kw, (o, lse, tol, tol_l) = paged_case(PAGED[i], 200 + i)
    got, got_l = attn.decode_paged(*args, return_lse=True, **kw)
    ref.check(got.transpose(1, 2), o, tol, "O")
    ref.check(got_l, lse, tol_l, "LSE")
    # a workspace full of NaN, and the same bits again
    ws = torch.full((1 << 22,), math.nan, device="cuda").view(torch.uint8)
    again, again_l = attn.decode_paged(*args, return_lse=True, workspace=ws, **kw)
    assert torch.equal(got.nan_to_num(7.0), again.nan_to_num(7.0)) and torch.equal(got_l, again_l)
    assert attn.attn_device_status() == attn.ATTN_OK


@pytest.mark.parametrize("dt,i8", [("bf16", False), ("f32", False), ("f16", True)])
@pytest.mark.parametrize("B,G,lens,window", [(1, 2, 700, None), (90, 8, 100, None), (70, 8, 500, None),
                                             (58, 8, 1900, None), (40, 4, 900, 70)])
def test_paged_writes_nothing_outside(dt, i8, B, G, lens, window):
    """The workspace the query asks for, the outputs, and not a byte beside them; every way of dividing the work."""
    g = gen(43)
    H, D, ps, guard = 2 * G, 64, 16, 4096
    n = torch.randint(0, lens + 1, (B,), generator=g).to(torch.int32)
    n[0] = lens
    width = -(-lens // ps)
    table = torch.randint(0, 50, (B, width), generator=g).to(torch.int32)
    if i8:
        k, v = (torch.randint(-128, 128, (50, G, ps, D), generator=g, dtype=torch.int8) for _ in range(2))
    else:
        k, v = randn(g, 50, G, ps, D, dt=DT[dt]), randn(g, 50, G, ps, D, dt=DT[dt])
    sc = [torch.rand(G * D, generator=g) * 0.015 + 0.005 for _ in range(2)]
    q = randn(g, B, 1, H, D, dt=DT[dt])
    qd, kd, vd, td, nd, ks, vs = (t.cuda() for t in (q, k, v, table, n, *sc))
    buf = torch.full((B * H * D + 2 * guard,), 7.0, dtype=DT[dt], device="cuda")
    out = buf[guard:-guard].view(B, 1, H, D)
    d = dict(batch=B, heads=H, kv_heads=G, q_len=1, k_len=lens, head_dim=D, dtype=dt, causal=window is not None,
             causal_align="klens", window_left=window, masked_rows="zero", k_layout=attn._layout4(kd, 1),
             v_layout=attn._layout4(vd, 1), q_layout=attn._layout4(qd, 2), o_layout=attn._layout4(out, 2))
    if i8:
        d.update(kv_dtype="i8", kv_scale="channel", k_scale_ptr=ks.data_ptr(), v_scale_ptr=vs.data_ptr())
    p, pages = attn.make_problem(d), attn.make_pages(ps, 50, td.data_ptr(), td.stride(0))
    size = attn.attn_decode_paged_workspace_size(p, pages, 0)
    ws = torch.full((size + 2 * guard * 64,), 171, dtype=torch.uint8, device="cuda")
    assert attn.attn_decode_paged(p, pages, 0, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), out.data_ptr(), None,
                                  nd.data_ptr(), None, ws.data_ptr() + guard * 64, size,
                                  torch.cuda.current_stream().cuda_stream) == 0
    rk, rv = ref.gather(k, table, ps, lens, False)[0], ref.gather(v, table, ps, lens, False)[0]
    vis = ref.visible(1, lens, n, window=-1 if window is None else window)
    o, _, tol, _ = ref.attention(q.transpose(1, 2), rk, rv, vis, kv_scales=sc if i8 else None, half_q=i8)
    ref.check(out.transpose(1, 2), o, tol)
    assert (buf[:guard] == 7).all() and (buf[-guard:] == 7).all()
    assert (ws[:guard * 64] == 171).all() and (ws[guard * 64 + size:] == 171).all()


def test_paged_matches_the_contiguous_decode_and_shares_pages():
    """The rows of one entry as pages of a pool, two entries naming the same pages."""
    g = gen(5)
    k, v = randn(g, 1, 2, 640, 128, dt=torch.bfloat16), randn(g, 1, 2, 640, 128, dt=torch.bfloat16)
    q = randn(g, 2, 1, 8, 128, dt=torch.bfloat16)
    pool = [t.view(2, 20, 32, 128).transpose(0, 1).contiguous().cuda() for t in (k, v)]
    table = torch.arange(20, dtype=torch.int32).repeat(2, 1).cuda()
    lens = torch.tensor([640, 321], dtype=torch.int32).cuda()
    got = attn.decode_paged(q.cuda(), *pool, table, lens)
    plain = attn.decode(q.cuda(), k.expand(2, -1, -1, -1).contiguous().cuda(),
                        v.expand(2, -1, -1, -1).contiguous().cuda(), lens)
    vis = ref.visible(1, 640, [640, 321])
    o, _, tol, _ = ref.attention(q.transpose(1, 2), k.expand(2, -1, -1, -1), v.expand(2, -1, -1, -1), vis)
    ref.check(got.transpose(1, 2), o, tol)
    ref.check(plain.transpose(1, 2), o, tol)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_paged_non_finite_scores(dt):
    """A visible NaN or +inf key makes its heads' rows NaN and no others; an infinite key that is hidden does nothing."""
    g = gen(9)
    k, v = randn(g, 40, 2, 16, 64, dt=DT[dt]), randn(g, 40, 2, 16, 64, dt=DT[dt])
    table = torch.arange(40, dtype=torch.int32).view(2, 20)
    q = randn(g, 2, 1, 4, 64, dt=DT[dt]).abs()
    k[3, 0, 5] = math.nan          # entry 0, kv head 0
    k[25, 1, 2] = math.inf         # entry 1, kv head 1: scores +inf
    k[19, 1, 15] = math.inf        # entry 0, behind its length
    got = attn.decode_paged(q.cuda(), k.cuda(), v.cuda(), table.cuda(),
                            torch.tensor([319, 320], dtype=torch.int32).cuda()).cpu()
    assert torch.isnan(got[0, 0, :2]).all() and torch.isfinite(got[0, 0, 2:]).all()
    assert torch.isnan(got[1, 0, 2:]).all() and torch.isfinite(got[1, 0, :2]).all()


def test_paged_offsets_past_32_bits():
    """Pages behind the first 2^31 elements of a pool."""
    n, ps, G, D = 2 ** 31 // (64 * 2 * 128) + 40, 64, 2, 128
    k = torch.zeros(n, G, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = gen(4)
    tail_k, tail_v = randn(g, 3, G, ps, D, dt=torch.bfloat16), randn(g, 3, G, ps, D, dt=torch.bfloat16)
    k[-3:], v[-3:] = tail_k.cuda(), tail_v.cuda()
    table = torch.tensor([[n - 1, n - 3, n - 2]], dtype=torch.int32)
    q = randn(g, 1, 1, 4, D, dt=torch.bfloat16)
    got = attn.decode_paged(q.cuda(), k, v, table.cuda(), torch.tensor([190], dtype=torch.int32).cuda())
    rows = [t[[2, 0, 1]].transpose(0, 1).reshape(1, G, 192, D) for t in (tail_k, tail_v)]
    o, _, tol, _ = ref.attention(q.transpose(1, 2), *rows, ref.visible(1, 192, [190]))
    ref.check(got.transpose(1, 2), o, tol)
    # and the write of a cache row there
    out = attn.qkv_prep(q, q[:, :, :2], q[:, :, 2:], k, v, table.cuda(), norm=False,
                        rows=torch.tensor([[70]], dtype=torch.int32).cuda()) if q.is_cuda else \
        attn.qkv_prep(q.cuda(), q[:, :, :2].cuda(), q[:, :, 2:].cuda(), k, v, table.cuda(), norm=False,
                      rows=torch.tensor([[70]], dtype=torch.int32).cuda())
    assert torch.equal(out.cpu(), q)
    assert torch.equal(k[n - 3, :, 6].cpu(), q[0, 0, :2]) and torch.equal(v[n - 3, :, 6].cpu(), q[0, 0, 2:])


# ---- norm, rotation and cache write ----------------------------------------------------------------

# dtype, D, rot, B, S, H, G, page_size (0: contiguous), options
PREP = [
    ("bf16", 128, 128, 3, 5, 8, 2, 16, {}),
    ("f16", 64, 64, 2, 130, 6, 3, 0, {}),
    ("f32", 64, 32, 2, 7, 4, 2, 8, dict(inter=True)),
    ("bf16", 128, 64, 1, 1, 2, 2, 24, dict(nhd=True)),
    ("f16", 256, 256, 2, 3, 4, 1, 5, dict(inter=True, nhd=True)),
    ("bf16", 256, 0, 2, 3, 2, 1, 16, {}),                                # no rotation
    ("f32", 256, 64, 1, 9, 2, 2, 0, {}),
    ("bf16", 80, 40, 2, 4, 3, 1, 16, {}),
    ("f32", 5, 4, 2, 4, 2, 1, 3, {}),
    ("f16", 96, 24, 2, 4, 3, 3, 16, dict(inter=True)),
    ("bf16", 128, 4, 2, 4, 3, 1, 16, {}),
    ("bf16", 128, 128, 2, 4, 4, 2, 16, dict(norm=False)),
    ("bf16", 64, 64, 2, 4, 4, 2, 16, dict(unit=True)),                   # norm without weights
    ("f16", 128, 128, 2, 6, 4, 2, 16, dict(i8="channel")),
    ("f32", 64, 64, 2, 6, 4, 2, 0, dict(i8="tensor")),
    ("bf16", 80, 80, 2, 6, 4, 2, 7, dict(i8="channel")),
    ("bf16", 128, 128, 2, 4, 4, 2, 16, dict(odd=1)),                     # rows that start off 16 bytes
    ("f32", 128, 128, 2, 4, 4, 2, 0, dict(odd=3)),
    ("bf16", 128, 128, 2, 4, 4, 2, 16, dict(inplace=True)),
    ("f32", 80, 64, 2, 4, 4, 2, 16, dict(inplace=True)),
    ("bf16", 64, 64, 300, 1, 4, 2, 16, {}),
    ("bf16", 128, 128, 1, 2, 70, 70, 0, {}),
]


def prep_case(c, seed):
    dt, D, rot, B, S, H, G, ps, opt = c
    g, dt = gen(seed), DT[dt]
    odd = opt.get("odd", 0)
    flat = randn(g, B * S * (H + 2 * G) * D + odd, dt=dt, scale=2.0)
    qkv = flat[odd:].view(B, S, H + 2 * G, D)
    qkv[0, 0, 0] = 0   # a head of zeros
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dt) for _ in range(2)]
    cap = S + 20
    ang = torch.arange(cap + 3, dtype=torch.float64)[:, None] * 100.0 ** -torch.linspace(0, 1, max(rot // 2, 1),
                                                                                         dtype=torch.float64)
    cos, sin = ang.cos().float(), ang.sin().float()
    pos = torch.randint(0, cap + 3, (B, S), generator=g).to(torch.int32)
    pos[0, 0], pos[-1, -1] = -5, 10 ** 6   # clamped to the tables
    row = torch.stack([torch.randperm(cap, generator=g)[:S] for _ in range(B)]).to(torch.int32)
    if S > 2:
        row[0, 1], row[-1, 2] = -1, cap   # tokens that write nothing
    nhd, width = opt.get("nhd", False), -(-cap // ps) if ps else 1
    table = torch.randperm(B * width + 2, generator=g)[:B * width].view(B, width).to(torch.int32)
    if ps:
        table[-1, -1] = -1
    shape = ((B * width + 2, ps, G, D) if nhd else (B * width + 2, G, ps, D)) if ps else (B, G, cap, D)
    cdt = torch.int8 if opt.get("i8") else dt
    kc, vc = (torch.randint(-9, 9, shape, generator=g).to(cdt) for _ in range(2))
    scales = [torch.rand(G * D if opt["i8"] == "channel" else 1, generator=g) * 0.02 + 0.02 for _ in range(2)] \
        if opt.get("i8") else None
    return dict(dt=dt, D=D, rot=rot, B=B, S=S, H=H, G=G, ps=ps, opt=opt, flat=flat, odd=odd, qkv=qkv, w=w, cos=cos,
                sin=sin, pos=pos, row=row, cap=width * ps if ps else cap, table=table, kc=kc, vc=vc, scales=scales,
                nhd=nhd)


def cache_targets(c):
    """For each token that writes: (b, i, outer index, row)."""
    out = []
    for b in range(c["B"]):
        for i in range(c["S"]):
            r = int(c["row"][b, i])
            if not 0 <= r < c["cap"]:
                continue
            page, at = (int(c["table"][b, r // c["ps"]]), r % c["ps"]) if c["ps"] else (b, r)
            if 0 <= page < c["kc"].shape[0]:
                out.append((b, i, page, at))
    return out


@pytest.mark.parametrize("i", range(len(PREP)))
def test_prep(i):
    c = prep_case(PREP[i], 300 + i)
    opt, H, G, dt = c["opt"], c["H"], c["G"], c["dt"]
    norm, inter = opt.get("norm", True), opt.get("inter", False)
    w = [None, None] if opt.get("unit") or not norm else c["w"]
    pos = c["pos"].long().clamp(0, c["cos"].shape[0] - 1)
    kw = dict(eps=1e-5, norm=norm, rot=c["rot"], inter=inter)
    q, tq = ref.prep(c["qkv"][:, :, :H], w[0], c["cos"], c["sin"], pos, **kw)
    k, tk = ref.prep(c["qkv"][:, :, H:H + G], w[1], c["cos"], c["sin"], pos, **kw)
    v = c["qkv"][:, :, H + G:].double()
    kc, vc = c["kc"].cuda(), c["vc"].cuda()
    qkv = c["flat"].cuda()[c["odd"]:].view(c["qkv"].shape)
    rot = dict(cos=c["cos"].cuda(), sin=c["sin"].cuda()) if c["rot"] else {}
    args = dict(q_weight=None if w[0] is None else w[0].cuda(), k_weight=None if w[1] is None else w[1].cuda(),
                eps=1e-5, norm=norm, interleaved=inter, positions=c["pos"].cuda(), rows=c["row"].cuda(),
                page_layout="nhd" if c["nhd"] else "hnd", **rot)
    if c["scales"]:
        args.update(k_scale=c["scales"][0].cuda(), v_scale=c["scales"][1].cuda())
    qin = qkv[:, :, :H]
    out = attn.qkv_prep(qin, qkv[:, :, H:H + G], qkv[:, :, H + G:], kc, vc, c["table"].cuda() if c["ps"] else None,
                        out=qin if opt.get("inplace") else None, **args)
    if opt.get("inplace"):
        assert torch.equal(qkv[:, :, H:].cpu(), c["qkv"][:, :, H:])   # K and V as they were
    ref.check(out, q, tq * 1.01 + ref.HALF[dt] * q.abs() + 2.0 ** -25, "q")
    # the caches: written rows by value, all others as they were
    sel = (lambda t, page, at: t[page, at] if c["nhd"] else t[page, :, at])
    want_k, want_v = c["kc"].double(), c["vc"].double()
    tol_k, tol_v = torch.zeros_like(want_k), torch.zeros_like(want_v)
    for b, t, page, at in cache_targets(c):
        for want, tol, x, e, s in ((want_k, tol_k, k, tk, 0), (want_v, tol_v, v, None, 1)):
            y = x[b, t]
            if c["scales"]:
                sc = c["scales"][s].double()
                y = y / (sc.view(G, -1) if sc.numel() > 1 else sc)
                err = 0 if e is None else e[b, t] / (sc.view(G, -1) if sc.numel() > 1 else sc)
                sel(want, page, at)[:] = y.clamp(-128, 127)
                sel(tol, page, at)[:] = 0.5 + err + y.abs() * 2.0 ** -23   # a code is off by half a step at most
            else:
                sel(want, page, at)[:] = y
                sel(tol, page, at)[:] = 0 if e is None else e[b, t] * 1.01 + ref.HALF[dt] * y.abs() + 2.0 ** -25
    ref.check(kc, want_k, tol_k, "k cache")
    ref.check(vc, want_v, tol_v, "v cache")


def test_prep_defaults_are_the_tokens_index():
    c = prep_case(("bf16", 128, 128, 2, 6, 4, 2, 0, {}), 7)
    qkv, idx = c["qkv"].cuda(), torch.arange(6, dtype=torch.int32).repeat(2, 1).cuda()
    kw = dict(cos=c["cos"].cuda(), sin=c["sin"].cuda())
    got = []
    for more in ({}, dict(positions=idx, rows=idx)):
        kc, vc = torch.zeros_like(c["kc"].cuda()), torch.zeros_like(c["vc"].cuda())
        got.append((attn.qkv_prep(qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:], kc, vc, **kw, **more), kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---- the three together ----------------------------------------------------------------------------


def serve(H, G, D, ps, prompts, steps, w, first, dt, graph=False):
    """A layer as a served model runs it: prepare and attend the prompts, then `steps` single tokens."""
    g = gen(11)
    B, S = len(prompts), max(prompts)
    cap = S + steps
    width = -(-cap // ps)
    cos = torch.randn(cap, D // 2, generator=g).cos().cuda()
    sin = torch.randn(cap, D // 2, generator=g).sin().cuda()
    table = torch.randperm(B * width, generator=g).view(B, width).to(torch.int32).cuda()
    kc, vc = (torch.zeros(B * width, G, ps, D, dtype=dt, device="cuda") for _ in range(2))
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).to(dt).cuda() for _ in range(2))
    n = torch.tensor(prompts, dtype=torch.int32).cuda()
    i = torch.arange(S, dtype=torch.int32, device="cuda")[None]
    at = torch.where(i < n[:, None], i, -1)
    common = dict(q_weight=qw, k_weight=kw, cos=cos, sin=sin)
    x = randn(g, B, S, H + 2 * G, D, dt=dt).cuda()
    # the prompt: contiguous copies for the windowed attention, pages for the steps
    kp, vp = (torch.zeros(B, G, S, D, dtype=dt, device="cuda") for _ in range(2))
    split = (lambda t: (t[:, :, :H], t[:, :, H:H + G], t[:, :, H + G:]))
    attn.qkv_prep(*split(x), kc, vc, table, positions=at, rows=at, **common)
    q = attn.qkv_prep(*split(x), kp, vp, positions=at, rows=at, **common)
    lens = n.clone()
    po = attn.fwd(q.transpose(1, 2), kp, vp, layout="bhsd", causal=True, causal_offset=0, k_lens=lens,
                  window_left=w, first_keys=first, masked_rows="zero")
    outs, seen = [], []
    xs = [randn(g, B, 1, H + 2 * G, D, dt=dt).cuda() for _ in range(steps)]
    xin, pos = torch.empty_like(xs[0]), torch.empty(B, 1, dtype=torch.int32, device="cuda")
    bufs = dict(out=torch.empty(B, 1, H, D, dtype=dt, device="cuda"))
    qbuf = torch.empty_like(bufs["out"])
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def step():
        pos.copy_(lens[:, None])
        attn.qkv_prep(*split(xin), kc, vc, table, positions=pos, rows=pos, out=qbuf, **common)
        lens.add_(1)
        attn.decode_paged(qbuf, kc, vc, table, lens, window_left=w, first_keys=first, workspace=ws,
                          masked_rows="zero", **bufs)

    run = step
    if graph:
        keep = [t.clone() for t in (lens, kc, vc)]
        xin.copy_(xs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for t, s in zip((lens, kc, vc), keep):
            t.copy_(s)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        run = cg.replay
    for s in range(steps):
        xin.copy_(xs[s])
        run()
        outs.append(bufs["out"].clone())
        seen.append((qbuf.clone(), lens.clone()))
    return dict(q=q, kp=kp, vp=vp, po=po, kc=kc, vc=vc, table=table, outs=outs, seen=seen, x=x, xs=xs, prompts=prompts,
                cos=cos, sin=sin, qw=qw, kw=kw)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_serving_run(dt):
    H, G, D, ps, w, first, steps, prompts = 4, 2, 64, 16, 40, 5, 7, [130, 77, 1]
    r = serve(H, G, D, ps, prompts, steps, w, first, DT[dt])
    cpu = (lambda t: t.detach().cpu())
    S = max(prompts)
    # the prompt's queries against the formula, its attention against the reference on what was stored
    pos = torch.where(torch.arange(S)[None] < torch.tensor(prompts)[:, None], torch.arange(S)[None], 0)
    q, tq = ref.prep(cpu(r["x"])[:, :, :H], cpu(r["qw"]), cpu(r["cos"]), cpu(r["sin"]), pos, eps=1e-6, norm=True,
                     rot=D, inter=False)
    ref.check(r["q"], q, tq * 1.01 + ref.HALF[DT[dt]] * q.abs() + 2.0 ** -25, "prompt q")
    vis = ref.visible(S, S, prompts, offset=0, window=w, first=first)
    o, _, tol, _ = ref.attention(cpu(r["q"]).transpose(1, 2), cpu(r["kp"]), cpu(r["vp"]), vis)
    ref.check(r["po"], o, tol, "prompt O")
    # each step against the rows in the pages
    for s, (out, (qs, lens)) in enumerate(zip(r["outs"], r["seen"])):
        rows = S + steps
        k, _ = ref.gather(cpu(r["kc"]), cpu(r["table"]), ps, rows, False)
        v, _ = ref.gather(cpu(r["vc"]), cpu(r["table"]), ps, rows, False)
        assert lens.tolist() == [p + s + 1 for p in prompts]
        vis = ref.visible(1, rows, lens.cpu(), window=w, first=first)
        o, _, tol, _ = ref.attention(cpu(qs).transpose(1, 2), k, v, vis)
        ref.check(out.transpose(1, 2), o, tol, f"step {s}")
    # the pages hold the prompt's rows
    for b, n in enumerate(prompts):
        k, _ = ref.gather(cpu(r["kc"]), cpu(r["table"]), ps, n, False)
        assert torch.equal(k[b], cpu(r["kp"])[b, :, :n])


def test_serving_run_captured_gives_the_same_bits():
    a = serve(4, 2, 128, 16, [300, 40], 5, 100, 4, torch.bfloat16)
    b = serve(4, 2, 128, 16, [300, 40], 5, 100, 4, torch.bfloat16, graph=True)
    for x, y in zip(a["outs"], b["outs"]):
        assert torch.equal(x, y)
    assert torch.equal(a["kc"], b["kc"]) and torch.equal(a["vc"], b["vc"])


def test_other_streams_and_offsets_of_views():
    """A call on a stream of its own, on views that start inside larger tensors."""
    g = gen(21)
    pool = randn(g, 12, 2, 2, 16, 128, dt=torch.float16).cuda()   # K and V of a page side by side
    table = torch.arange(12, dtype=torch.int32).view(2, 6).cuda()
    lens = torch.tensor([90, 33], dtype=torch.int32).cuda()
    big = randn(g, 2, 3, 4, 128, dt=torch.float16).cuda()
    q = big[:, 1:2]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = attn.decode_paged(q, pool[:, 0], pool[:, 1], table, lens)
    st.synchronize()
    k, _ = ref.gather(pool[:, 0].cpu(), table.cpu(), 16, 96, False)
    v, _ = ref.gather(pool[:, 1].cpu(), table.cpu(), 16, 96, False)
    o, _, tol, _ = ref.attention(q.cpu().transpose(1, 2), k, v, ref.visible(1, 96, [90, 33]))
    ref.check(got.transpose(1, 2), o, tol)


def test_two_streams_at_once():
    """Calls that run side by side, each with its own outputs and workspace, give what they give alone."""
    jobs = [paged_case(PAGED[i], 400 + i) for i in (len(PAGED) - 10, 1)] + [paged_case(PAGED[0], 410)]
    want = [attn.decode_paged(*a, **kw) for a, kw, _ in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [[] for _ in jobs]
    for _ in range(10):
        for st, (a, kw, _), g in zip(streams, jobs, got):
            with torch.cuda.stream(st):
                g.append(attn.decode_paged(*a, **kw))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w.nan_to_num(3.0), x.nan_to_num(3.0)) for x in g)


def test_paged_many_entries():
    """Thousands of short entries, most without a key."""
    g = gen(41)
    B, G, ps, D = 3500, 1, 8, 64
    lens = torch.randint(-6, 4, (B,), generator=g).clamp(min=0)
    k, v = randn(g, B, G, ps, D, dt=torch.float16), randn(g, B, G, ps, D, dt=torch.float16)
    q = randn(g, B, 1, 2, D, dt=torch.float16)
    table = torch.arange(B, dtype=torch.int32).view(B, 1)
    got = attn.decode_paged(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.to(torch.int32).cuda(),
                            masked_rows="zero")
    o, _, tol, _ = ref.attention(q.transpose(1, 2), k, v, ref.visible(1, ps, lens))
    ref.check(got.transpose(1, 2), o, tol)


@pytest.mark.parametrize("dt,i8,D,H,G,B,rows,opt", [
    ("f16", None, 64, 8, 8, 58, 1800, dict(zero=False)),
    ("bf16", None, 128, 16, 8, 58, 900, dict(sink=True)),
    ("bf16", "channel", 128, 16, 8, 58, 1700, {}),
    ("f16", "tensor", 64, 24, 8, 59, 1800, dict(sink=True)),
    ("f32", None, 64, 16, 8, 58, 900, dict(softcap=15.0)),
    ("f32", None, 128, 64, 8, 39, 500, dict(sink=True)),
    ("bf16", None, 256, 16, 8, 20, 900, dict(zero=False)),
    ("bf16", None, 128, 72, 4, 39, 900, {}),
    ("f16", None, 64, 8, 8, 60, 2500, dict(window=1500, first=5)),
])
def test_paged_shares(dt, i8, D, H, G, B, rows, opt):
    """Lists too many and too long for clusters and whole units: cut anywhere, ends and empty entries among them."""
    g = gen(47)
    ps, w, first, zero = 16, opt.get("window", -1), opt.get("first", 0), opt.get("zero", True)
    long = torch.rand(B, generator=g) < 0.4
    n = torch.where(long, torch.randint(0, rows + 1, (B,), generator=g), torch.randint(0, 70, (B,), generator=g))
    n[torch.rand(B, generator=g) < 0.1] = 0
    n[B // 2] = rows
    width = -(-rows // ps)
    table = torch.randint(0, 60, (B, width), generator=g).to(torch.int32)
    if i8:
        k, v = (torch.randint(-128, 128, (60, G, ps, D), generator=g, dtype=torch.int8) for _ in range(2))
        sc = [torch.rand(G * D if i8 == "channel" else 1, generator=g) * 0.015 + 0.005 for _ in range(2)]
    else:
        k, v, sc = randn(g, 60, G, ps, D, dt=DT[dt]), randn(g, 60, G, ps, D, dt=DT[dt]), None
    q = randn(g, B, 1, H, D, dt=DT[dt])
    sink = randn(g, H) if opt.get("sink") else None
    kw = dict(masked_rows="zero" if zero else "nan", softcap=opt.get("softcap", 0.0), max_rows=rows,
              window_left=None if w < 0 else w, first_keys=first, head_sink=None if sink is None else sink.cuda())
    if i8:
        kw.update(k_scale=sc[0].cuda(), v_scale=sc[1].cuda())
    args = [t.cuda() for t in (q, k, v, table, n.to(torch.int32))]
    got, lse = attn.decode_paged(*args, return_lse=True, **kw)
    again = attn.decode_paged(*args, workspace=torch.full((1 << 22,), math.nan, device="cuda").view(torch.uint8), **kw)
    assert torch.equal(got.nan_to_num(7.0), again.nan_to_num(7.0))
    for b in range(B):
        m = max(int(n[b]), 1)
        rk, rv = (ref.gather(t, table[b:b + 1], ps, m, False)[0] for t in (k, v))
        vis = ref.visible(1, m, n[b:b + 1], window=w, first=first)
        o, l, tol, tol_l = ref.attention(q[b:b + 1].transpose(1, 2), rk, rv, vis, softcap=opt.get("softcap", 0.0),
                                         sink=sink, zero=zero, kv_scales=sc, half_q=bool(i8) and dt != "f32")
        ref.check(got[b:b + 1].transpose(1, 2), o, tol, f"O of entry {b}")
        ref.check(lse[b:b + 1], l, tol_l, f"LSE of entry {b}")


def test_python_entry_points_refuse():
    f = dict(device="cuda", dtype=torch.float16)
    q, pool = torch.zeros(2, 1, 4, 64, **f), torch.zeros(8, 2, 16, 64, **f)
    table, lens = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    good = dict(q=q, k_pool=pool, v_pool=pool, table=table, k_lens=lens)
    attn.decode_paged(**good)
    for bad in (dict(table=table.long()), dict(table=table.cpu()), dict(k_pool=pool.float()), dict(k_lens=lens.float()),
                dict(v_pool=pool[:, :1]), dict(table=table[:1]), dict(table=table[:, ::2]), dict(k_lens=lens[:1]),
                dict(v_pool=pool.to(torch.int8)), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            attn.decode_paged(**dict(good, **bad))
    with pytest.raises(ValueError):
        attn.decode_paged(**good, max_rows=65)
    with pytest.raises(attn.AttnError):
        attn.decode_paged(**good, first_keys=3)
    kc = torch.zeros(2, 2, 16, 64, **f)
    k = torch.zeros(2, 1, 2, 64, **f)
    cos = torch.zeros(8, 32, device="cuda")
    good = dict(q=q, k=k, v=k, k_cache=kc, v_cache=kc.clone(), cos=cos, sin=cos)
    attn.qkv_prep(**good)
    for bad in (dict(sin=None), dict(cos=cos.half()), dict(k=k.float()), dict(v=k[:, :, :1]), dict(k_cache=kc[:1]),
                dict(q_weight=torch.ones(32, **f)), dict(rows=torch.zeros(2, 2, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(2, 1, device="cuda")), dict(v_cache=kc.float())):
        with pytest.raises(ValueError):
            attn.qkv_prep(**dict(good, **bad))
    qq = torch.zeros(1, 2, 8, 64, **f)
    with pytest.raises(attn.AttnError):
        attn.fwd(qq, qq, qq, layout="bhsd", causal=True, first_keys=2)
    with pytest.raises(ValueError):
        attn.fwd(qq, qq.float(), qq, layout="bhsd", causal=True, window_left=2, first_keys=2)
