"""GPU parity of attn_fwd_shared against float64, at the lengths, sizes, lists,
layouts and transforms where it can go wrong."""
from __future__ import annotations

import math

import pytest

import serving_bounds as sb
import shared_cases as sc
from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert attn.attn_device_status(torch.cuda.current_stream().cuda_stream) == 0


# dtype, D, B, Sq, H, G, page size, prefix rows, own lengths, options
CASES = [
    ("bf16", 128, 4, 1, 8, 2, 16, 1000, [1, 100, 37, 64], {}),
    ("f16", 128, 3, 1, 8, 2, 64, 128, [0, 1, 200], {}),                                    # an entry without own keys
    ("bf16", 64, 2, 1, 12, 4, 24, 333, [5, 77], dict(nhd=True)),
    ("bf16", 64, 40, 1, 4, 4, 8, 2100, [(7 * i) % 131 for i in range(40)], {}),            # one head a kv head
    ("f16", 64, 70, 1, 8, 1, 16, 1501, [(11 * i) % 50 for i in range(70)], {}),            # more than two row tiles
    ("bf16", 128, 5, 1, 6, 2, 32, 0, [3, 0, 129, 64, 500], dict(masked_rows="zero")),      # no prefix, an empty row
    ("f16", 64, 3, 1, 4, 2, 16, 0, [3, 0, 12], {}),                                        # ... that gives NaN
    ("bf16", 128, 2, 1, 4, 2, 16, 700, [0, 0], dict(max_rows=0)),                          # a prefix alone
    ("bf16", 128, 9, 5, 8, 2, 16, 777, [5, 6, 30, 128, 4, 1, 0, 200, 131], {}),            # drafted tokens, short entries
    ("f16", 64, 3, 3, 6, 2, 16, 2000, [3, 90, 33], dict(nhd=True)),
    ("bf16", 128, 2, 130, 8, 2, 64, 300, [130, 400], {}),                                  # prompts
    ("f16", 128, 2, 300, 4, 1, 16, 129, [300, 150], {}),                                   # rows in front of the own keys
    ("bf16", 64, 1, 257, 3, 3, 128, 1, [600], {}),
    ("bf16", 128, 64, 1, 8, 8, 16, 3000, [(7 * i) % 131 for i in range(64)], dict(max_rows=3000)),  # much room, few keys
    ("f16", 64, 70, 1, 8, 8, 16, 5000, [(7 * i) % 131 for i in range(70)], dict(max_rows=9000)),
    ("bf16", 128, 3, 150, 8, 2, 16, 700, [150, 151, 160], dict(max_rows=5000)),
    ("f16", 64, 9, 12, 8, 2, 16, 3000, [12, 151, 0, 160, 1, 2, 3, 4, 5], dict(max_rows=4000)),
    ("bf16", 128, 2, 600, 8, 2, 64, 129, [600, 100], dict(max_rows=2000, offset=40)),
    ("f32", 64, 3, 40, 4, 2, 16, 300, [40, 41, 7], dict(max_rows=4000)),
    ("bf16", 64, 3, 70, 4, 4, 8, 500, [70, 71, 64], dict(causal=False)),
    ("f16", 128, 2, 40, 4, 2, 32, 260, [300, 40], dict(offset=100)),
    ("f16", 128, 2, 40, 4, 2, 32, 260, [300, 40], dict(offset=-20)),
    ("bf16", 128, 3, 20, 4, 2, 16, 0, [20, 10, 0], dict(masked_rows="zero")),
    ("bf16", 128, 4, 1, 8, 2, 32, 500, [10, 20, 300, 0], dict(softcap=2.0)),
    ("f16", 128, 3, 33, 8, 2, 16, 500, [33, 40, 50], dict(softcap=5.0, smooth_softmax=True)),
    ("bf16", 64, 3, 33, 8, 2, 16, 500, [33, 40, 50], dict(smooth_softmax=True, scale=-0.2)),
    ("bf16", 128, 3, 1, 8, 2, 16, 500, [33, 0, 50], dict(smooth_softmax=True, scale=0.3)),
    ("bf16", 64, 3, 1, 4, 2, 16, 300, [20, 64, 50], dict(holes=[(0, 0), (1, 2), (2, 3)], prefix_holes=[0, 7, 18])),
    ("f16", 128, 3, 50, 4, 2, 16, 300, [80, 64, 50], dict(holes=[(0, 0), (1, 2), (2, 3)], prefix_holes=[0, 7, 18])),
    ("bf16", 128, 2, 9, 4, 2, 8, 40, [9, 12], dict(prefix_holes=range(5), masked_rows="zero")),   # no page of the prefix
    ("bf16", 128, 2, 7, 4, 2, 16, 200, [9, 12], dict(pad=8)),
    ("bf16", 128, 2, 7, 4, 2, 16, 200, [9, 12], dict(pad=2)),                              # rows off the 16-byte boundaries
    ("f16", 64, 3, 1, 4, 2, 16, 200, [9, 12, 1], dict(pad=1 * 2)),
    ("bf16", 64, 2, 19, 4, 2, 16, 200, [30, 12], dict(bhsd=True)),
    ("bf16", 128, 3, 1, 4, 2, 5, 203, [9, 12, 0], {}),                                     # odd pages
    ("f16", 128, 3, 17, 4, 2, 7, 203, [19, 12, 0], {}),
    ("bf16", 128, 3, 1, 4, 2, 1, 61, [9, 12, 0], {}),
    ("bf16", 128, 3, 9, 4, 2, 1000, 1500, [9, 12, 0], {}),
    ("bf16", 256, 3, 1, 8, 2, 16, 500, [9, 120, 0], {}),
    ("f16", 256, 2, 12, 4, 2, 16, 130, [12, 70], {}),
    ("bf16", 80, 2, 12, 4, 2, 16, 130, [12, 70], {}),
    ("f16", 6, 2, 1, 4, 2, 16, 130, [12, 70], {}),
    ("f32", 64, 3, 1, 12, 4, 16, 501, [33, 0, 100], {}),
    ("f32", 64, 5, 33, 12, 4, 16, 501, [33, 40, 77, 100, 20], {}),
    ("f32", 128, 2, 70, 4, 2, 32, 129, [33, 200], dict(softcap=3.0)),
    ("f32", 33, 2, 3, 4, 2, 16, 129, [33, 2], {}),
    ("f32", 128, 33, 1, 8, 2, 24, 1000, [(5 * i) % 64 for i in range(33)], {}),
    ("f32", 256, 2, 9, 4, 2, 16, 77, [9, 12], {}),
    ("f32", 128, 60, 1, 16, 4, 16, 6003, [(5 * i) % 90 for i in range(60)], dict(softcap=4.0)),   # packed rows
    ("f32", 64, 70, 1, 8, 8, 7, 7003, [(3 * i) % 40 for i in range(70)], dict(smooth_softmax=True)),
    ("f32", 64, 20, 3, 8, 4, 16, 4001, [(5 * i) % 90 for i in range(20)], dict(prefix_holes=[3, 250], holes=[(19, 0)])),
    ("f32", 128, 3, 2, 2, 2, 24, 3001, [2, 7, 0], dict(nhd=True, pad=4)),
    ("bf16", 128, 3, 1, 8, 2, 16, 400, [1, 50, 0], dict(i8="channel")),
    ("f16", 64, 3, 1, 8, 2, 16, 400, [1, 50, 0], dict(i8="tensor")),
    ("bf16", 128, 2, 6, 8, 2, 16, 100, [6, 50], dict(i8="channel")),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_shared(i):
    dt, D, B, Sq, H, G, ps, prefix, lens, opt = CASES[i]
    c = sc.make(dt, D, B, Sq, H, G, ps, prefix, lens, 900 + i, **opt)
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse, str(CASES[i]), **(dict(extra_score=2.0 ** -22) if opt.get("i8") else {}))


@pytest.mark.parametrize("dt,D,Sq", [("bf16", 128, 1), ("f16", 64, 1), ("bf16", 64, 40), ("f16", 128, 40), ("f32", 64, 1),
                                     ("f32", 64, 40), ("f16", 128, 5)])
@pytest.mark.parametrize("shape", ["bhqk", "1h1k", "b11k"])
def test_masks(dt, D, Sq, shape):
    """Ordinary, lowest, infinite and large masks, over the concatenated keys."""
    B, H, G, prefix, lens = 5, 4, 2, 300, [Sq, Sq + 30, 2 * Sq, Sq + 111, max(Sq - 2, 0)]
    g = torch.Generator(device="cuda")
    g.manual_seed(D + Sq)
    dims = {"bhqk": (B, H, Sq), "1h1k": (1, H, 1), "b11k": (B, 1, 1)}[shape]
    mask = sb.mask_kinds(g, *dims, prefix + max(lens))
    c = sc.make(dt, D, B, Sq, H, G, 16, prefix, lens, 7, mask=mask, masked_rows="zero")
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Sq", [1, 30])
def test_masks_of_nan_and_infinity(dt, Sq):
    """A mask of NaN or +inf on a visible key makes its row NaN and no other; on hidden keys it does nothing."""
    B, H, G, prefix, lens = 3, 4, 2, 200, [Sq + 9, Sq, Sq + 40]
    c = sc.make(dt, 128, B, Sq, H, G, 16, prefix, lens, 3)
    vis = c["ref"][3]
    mask = torch.where(vis[:, None], 0.0, math.nan).expand(B, H, Sq, -1).contiguous()
    mask[1, 2, 0, 7] = math.nan
    mask[2, 1, Sq - 1, prefix] = math.inf
    out, lse = sc.run(c, mask=mask, return_lse=True)
    bad = torch.zeros(B, Sq, H, dtype=torch.bool, device="cuda")
    bad[1, 0, 2] = bad[2, Sq - 1, 1] = True
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad.transpose(1, 2))
    clean = torch.where(torch.isfinite(mask), mask, 0.0)
    want = sc.run(c, mask=clean)
    assert torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("dt,Sq", [("bf16", 1), ("f16", 1), ("bf16", 20), ("f16", 20), ("f32", 20)])
def test_sinks(dt, Sq):
    H = 6
    sink = torch.tensor([0.0, 3.0, -math.inf, -50.0, 60.0, 1.0], device="cuda")
    c = sc.make(dt, 64, 3, Sq, H, 2, 16, 300, [Sq, Sq + 3, 0], 5, head_sink=sink)
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse)
    c["args"]["head_sink"] = torch.tensor([0.0, math.nan, 1.0, math.inf, 0.0, 0.0], device="cuda")
    out, lse = sc.run(c, return_lse=True)
    bad = torch.tensor([False, True, False, True, False, False], device="cuda")
    assert torch.equal(torch.isnan(lse).all(-1).all(0), bad) and torch.isnan(out[:, :, bad]).all()
    assert not torch.isnan(out[:, :, ~bad]).any()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("Sq", [1, 25])
@pytest.mark.parametrize("step", [4.0, -4.0])
def test_climbing_scores(dt, Sq, step):
    """Scores that climb (or fall) from tile to tile by more than a reference may lag."""
    c = sc.make(dt, 64, 3, Sq, 4, 2, 16, 900, [Sq + 200, Sq, Sq + 17], 11)
    q, k, v, ptab, prefix, table = c["call"]
    q.abs_()
    q[..., 1:] *= 0.05
    ramp = (torch.arange(prefix, device="cuda") // 128).to(k.dtype) * step
    r = torch.arange(prefix, device="cuda")
    k[ptab[r // 16].long(), :, r % 16, 0] = ramp[:, None] * 8
    c["ref"][1][:, :, :prefix, 0] = ramp * 8
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse)


@pytest.mark.parametrize("dt,Sq,B", [("bf16", 1, 6), ("f16", 5, 20), ("bf16", 150, 2), ("f32", 1, 6), ("f32", 20, 3), ("f32", 1, 70)])
def test_writes_nothing_outside(dt, Sq, B):
    """Outputs with gaps, a guarded workspace, and pools that stay as they were."""
    H, D = 8, 128
    c = sc.make(dt, D, B, Sq, H, 2, 16, 700, [Sq + 3 * b for b in range(B)], 21)
    q, k, v = c["call"][:3]
    ks, vs = k.clone(), v.clone()
    T = q.dtype
    flat = torch.full((B, Sq + 1, H + 1, D + 8), 7.0, dtype=T, device="cuda")
    out = flat[:, :Sq, :H, :D]
    lse_flat = torch.full((B, H + 1, Sq), 7.0, device="cuda")
    lse = lse_flat[:, :H]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    probe = sc.run(c)   # (the size that the library asks for is taken by the call without a workspace)
    sc.run(c, out=out, lse=lse, workspace=ws)
    assert torch.equal(out, probe)
    mark = torch.zeros_like(flat, dtype=torch.bool)
    mark[:, :Sq, :H, :D] = True
    assert (flat[~mark] == 7).all() and (lse_flat[:, H:] == 7).all()
    same = lambda a, b: torch.equal(torch.nan_to_num(a, nan=9.0), torch.nan_to_num(b, nan=9.0))  # noqa: E731
    assert same(k, ks) and same(v, vs)


@pytest.mark.parametrize("dt,Sq,B", [("bf16", 1, 30), ("bf16", 5, 20), ("f16", 200, 2), ("f32", 1, 9), ("f32", 1, 90), ("f32", 20, 3)])
def test_captured_replayed_and_on_other_streams(dt, Sq, B):
    """Two captured graphs that share a workspace, replayed in turn, and a call on another stream: the same bits."""
    cs = [sc.make(dt, 64, B, Sq, 8, 2, 16, 1300, [Sq + (5 * b + s) % 60 for b in range(B)], 31 + s) for s in range(2)]
    want = [sc.run(c) for c in cs]
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(w) for w in want], []
    for c, o in zip(cs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sc.run(c, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for i, st in enumerate(streams):   # side by side, each with its own workspace
            got[i] = sc.run(cs[i], stream=st.cuda_stream)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o, w)


def test_one_entry_is_the_paged_decode_of_both_lists():
    """The prefix in whole pages in front of an entry's own list: attn_decode_paged over the joined lists."""
    c = sc.make("bf16", 128, 6, 1, 8, 2, 16, 640, [1, 30, 16, 7, 64, 0], 41)
    q, k, v, ptab, prefix, table = c["call"]
    joined = torch.cat([ptab.expand(6, -1), table], 1).contiguous()
    want = attn.decode_paged(q, k, v, joined, c["args"]["k_lens"] + prefix, max_rows=prefix + c["args"]["max_rows"])
    got = sc.run(c)
    assert (got.float() - want.float()).abs().max() < 0.02


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements: pages behind it in the prefix's and the entries' lists."""
    ps, G, D = 64, 2, 128
    n_pages = 2 ** 32 // (ps * G * D) + 40
    k = torch.empty(n_pages, G, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    last = torch.arange(n_pages - 12, n_pages, dtype=torch.int32, device="cuda")
    for t in (k, v):
        t[-12:] = torch.randn(12, G, ps, D, device="cuda").to(t.dtype)
    for Sq, B in ((1, 2), (70, 2)):
        q = torch.randn(B, Sq, 4, D, device="cuda").to(k.dtype)
        n = torch.tensor([100, 128], dtype=torch.int32, device="cuda")
        table = last[8:].view(2, 2).contiguous()
        out = attn.fwd_shared(q, k, v, last[:8].contiguous(), 500, table, n)
        near = attn.fwd_shared(q, k[-12:].contiguous(), v[-12:].contiguous(), last[:8] - (n_pages - 12), 500,
                               table - (n_pages - 12), n)
        assert torch.equal(out, near)


@pytest.mark.parametrize("dt,D,Sq,B", [("bf16", 128, 1, 100), ("f16", 64, 30, 2)])
def test_bounded_wait(dt, D, Sq, B):
    """A copy that never comes: the call gives up after its limit, reports it, and the next call is right."""
    c = sc.make(dt, D, B, Sq, 8, 8, 16, 8000, [Sq + 3 * b for b in range(B)], 61)
    st = torch.cuda.current_stream().cuda_stream
    want = sc.run(c)
    assert attn.attn_device_status(st) == attn.ATTN_OK
    assert attn.attn_test_inject(attn.ATTN_INJECT_DROP_FIRST_COPY) == attn.ATTN_OK
    sc.run(c)
    assert attn.attn_device_status(st) == attn.ATTN_ERR_DEVICE_TIMEOUT
    assert torch.equal(sc.run(c), want)


@pytest.mark.parametrize("dt,D,Sq,B,H,G,prefix", [
    ("f16", 64, 30, 2, 8, 8, 8000), ("bf16", 128, 9, 30, 8, 2, 900), ("bf16", 64, 1, 300, 16, 8, 3000),
    ("f16", 128, 140, 5, 8, 8, 700)])
def test_many_times_over(dt, D, Sq, B, H, G, prefix):
    """Items in which a row tile has nothing to do, again and again: no wait runs out, the bits stay."""
    c = sc.make(dt, D, B, Sq, H, G, 16, prefix, [Sq + (7 * b) % 200 for b in range(B)], 71)
    want = sc.run(c)
    sc.check(c, want)
    out = torch.empty_like(want)
    for _ in range(60):
        out.fill_(9.0)
        sc.run(c, out=out)
        assert torch.equal(out, want)
    assert attn.attn_device_status(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK


@pytest.mark.parametrize("dt,D,Sq,B,H,G,prefix", [
    ("bf16", 128, 1, 60, 8, 2, 4000), ("f16", 64, 1, 150, 8, 8, 3001), ("f16", 128, 4, 30, 8, 2, 3000),
    ("bf16", 64, 3, 40, 4, 4, 5003), ("f32", 64, 1, 70, 8, 8, 5000), ("f32", 128, 3, 20, 8, 4, 3001)])
@pytest.mark.parametrize("kind", ["mask", "sink", "cap"])
def test_transforms_behind_long_prefixes(dt, D, Sq, B, H, G, prefix, kind):
    """Masks, sinks and softcaps where the prefix is read once for all entries."""
    g = torch.Generator(device="cuda")
    g.manual_seed(D + Sq + B)
    lens, kw = [(7 * b) % 90 for b in range(B)], dict(masked_rows="zero")
    if kind == "mask":
        kw["mask"] = sb.mask_kinds(g, B, H, Sq, prefix + max(lens))
    elif kind == "sink":
        kw["head_sink"] = torch.linspace(-3.0, 8.0, H, device="cuda")
    else:
        kw["softcap"] = 3.0
    c = sc.make(dt, D, B, Sq, H, G, 16, prefix, lens, 81, **kw)
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse)


@pytest.mark.parametrize("dt,D,B,Sq,H,G,ps,prefix,short,full", [
    ("bf16", 128, 2, 73, 12, 4, 128, 20040, 55, 79),      # few units, many shares of each
    ("f16", 128, 2, 301, 8, 2, 32, 5288, 453, 624),
    ("bf16", 64, 8, 261, 16, 8, 32, 1894, 1615, 2297),
    ("f16", 64, 1, 471, 4, 1, 24, 119, 177, 1420),
    ("bf16", 128, 2, 805, 8, 4, 16, 3001, 800, 817),      # last blocks of one row tile
    ("f32", 64, 9, 2, 4, 2, 64, 11635, 237, 1611),        # own lists in parts
    ("f32", 128, 1, 4, 4, 1, 32, 20615, 13, 13),
    ("f32", 64, 77, 28, 2, 2, 32, 88, 348, 433),
    ("f32", 128, 5, 60, 8, 4, 24, 500, 61, 500)])
def test_cut_lists(dt, D, B, Sq, H, G, ps, prefix, short, full):
    """Lists that are cut among CTAs, with a sink and without: own lists from `short` to `full` keys."""
    lens = [short + (full - short) * b // max(B - 1, 1) for b in range(B)]
    for kw in ({}, dict(smooth_softmax=True)):
        c = sc.make(dt, D, B, Sq, H, G, ps, prefix, lens, 95, max_rows=full, **kw)
        out, lse = sc.run(c, return_lse=True)
        sc.check(c, out, lse)
        assert torch.equal(sc.run(c), out)


@pytest.mark.parametrize("dt,Sq,B,prefix", [("bf16", 1, 4, 200), ("f16", 1, 60, 4000), ("bf16", 30, 3, 400), ("f32", 9, 3, 200)])
def test_pages_named_more_than_once(dt, Sq, B, prefix):
    """A page twice in the prefix's list, in two entries' lists, and in both kinds of list."""
    c = sc.make(dt, 64, B, Sq, 8, 4, 16, prefix, [64] * B, 91, poison=False)
    q, k, v, ptab, _, table = c["call"]
    ptab[3] = ptab[1]
    table[1] = table[0]
    table[2, :2] = ptab[4:6]
    rows = [torch.cat([p[ptab.long()].transpose(1, 2).flatten(0, 1)[:prefix].expand(B, -1, -1, -1),
                       p[table.long()].transpose(2, 3).flatten(1, 2)], 1).transpose(1, 2) for p in (k, v)]
    c["ref"] = (c["ref"][0], *rows, c["ref"][3])
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse)


def test_refusals():
    c = sc.make("bf16", 128, 2, 3, 4, 2, 16, 100, [9, 12], 51)
    q, k, v, ptab, prefix, table = c["call"]
    for bad in (dict(prefix_rows=-1), dict(prefix_rows=ptab.numel() * 16 + 1), dict(prefix_table=ptab.long()),
                dict(prefix_table=ptab.cpu()), dict(prefix_table=ptab[None]), dict(max_rows=table.shape[1] * 16 + 1),
                dict(mask=torch.zeros(1, 1, 1, prefix, device="cuda")), dict(lse=torch.zeros(2, 4, 2, device="cuda")),
                dict(workspace=torch.empty(1 << 22, dtype=torch.uint8)), dict(k_pool=k.float()), dict(v_pool=v[:-1])):
        kw = dict(dict(q=q, k_pool=k, v_pool=v, prefix_table=ptab, prefix_rows=prefix, table=table), **bad)
        with pytest.raises((ValueError, attn.AttnError)):
            attn.fwd_shared(**kw)
    big = sc.make("bf16", 128, 40, 1, 8, 2, 16, 4000, [9] * 40, 52)
    with pytest.raises(attn.AttnError):
        sc.run(big, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
