"""Paged decode over lists whose weight lies on chosen keys, so that a lost or
repeated tile, a wrong page and a wrong fragment show at any length: very long
lists in many fragments, and every way of dividing the units over the CTAs."""
from __future__ import annotations

import pytest

import serving_bounds as sb
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


def run(dt, D, H, G, ps, lens, marked, i8=False, nhd=False, seed=1, mask=False, window=-1, first=0):
    """Every entry has `marked` keys of high scores, at its first and last rows and spread between."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, rows = len(lens), max(lens)
    width = -(-rows // ps)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    counts = [-(-n // ps) for n in lens]
    n_pages = sum(counts) + 1
    perm = torch.randperm(n_pages - 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), n_pages - 1, dtype=torch.int32, device="cuda")   # (the last page: not to be used)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    q = rand(B, 1, H, D).to(DT[dt])
    u = q[:, 0].view(B, G, H // G, D)[:, :, 0].float()
    u = u / u.norm(dim=-1, keepdim=True)
    shape = (n_pages, G, ps, D)
    sc = None
    if i8:
        k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
        k //= 8
        sc = [torch.full((G * D,), 0.05, device="cuda"), torch.rand(G * D, generator=g, device="cuda") * 0.01 + 0.01]
    else:
        k, v = rand(*shape).to(DT[dt]), rand(*shape).to(DT[dt])
    for b, n in enumerate(lens):
        if n == 0:
            continue
        r = torch.linspace(0, n - 1, min(marked, n), device="cuda").round().long()
        r[1:-1] = (r[1:-1] + torch.randint(-20, 21, r[1:-1].shape, generator=g, device="cuda")).clamp(0, n - 1)
        page = table[b, r // ps].long()
        lifted = k[page, :, r % ps].float() * (0.05 if i8 else 1) + 25 * u[b]
        k[page, :, r % ps] = ((lifted / 0.05).round().clamp(-128, 127).to(torch.int8) if i8 else lifted.to(DT[dt]))
    k[-1], v[-1] = (127, 127) if i8 else (float("nan"), float("nan"))
    pools = [t.transpose(1, 2).contiguous() if nhd else t for t in (k, v)]
    m = rand(B, H, 1, rows) if mask else None
    kw = dict(k_scale=sc[0], v_scale=sc[1]) if i8 else {}
    got, lse = attn.decode_paged(q, *pools, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), max_rows=rows,
                                 page_layout="nhd" if nhd else "hnd", masked_rows="zero", return_lse=True, mask=m,
                                 window_left=None if window < 0 else window, first_keys=first, **kw)
    for b, n in enumerate(lens):
        if n == 0:
            assert (got[b] == 0).all() and (lse[b] == -float("inf")).all()
            continue
        j = torch.arange(n, device="cuda")
        vis = (j >= 0 if window < 0 else (j >= n - 1 - window) | (j < first))[None, None]
        kk, vv = (sb.rows_of(t, table[b:b + 1], ps, n) for t in (k, v))
        o, l, tol, tol_l = sb.attention(q[b:b + 1].transpose(1, 2), kk, vv, vis, kv_scales=sc,
                                        mask=None if m is None else m[b:b + 1, :, :, :n],
                                        extra_score=2.0 ** -22 if i8 else 0.0)
        sb.check(got[b:b + 1].transpose(1, 2), o, tol, f"O of entry {b}")
        sb.check(lse[b:b + 1], l, tol_l, f"LSE of entry {b}")


@pytest.mark.parametrize("dt,D,H,G,ps,lens,opt", [
    ("bf16", 128, 4, 1, 64, [131072], {}),                      # one unit in hundreds of fragments
    ("f16", 128, 8, 2, 32, [131072, 100001], dict(nhd=True)),
    ("f16", 64, 3, 1, 16, [130001], dict(mask=True)),
    ("f32", 64, 2, 1, 24, [100003, 77], {}),
    ("f32", 128, 8, 1, 64, [65537], {}),
    ("bf16", 128, 8, 2, 64, [99999, 1, 0], dict(i8=True)),
    ("f16", 64, 16, 1, 128, [120000], dict(i8=True)),
    ("bf16", 256, 4, 1, 16, [70001], {}),
    ("bf16", 64, 4, 2, 16, [90000, 70000], dict(window=60000, first=900)),
])
@pytest.mark.parametrize("marked", [7, 300])
def test_long_lists(dt, D, H, G, ps, lens, opt, marked):
    run(dt, D, H, G, ps, lens, marked, **opt)


# With bf16 at head_dim 128 an SM has three CTAs: a unit gets the most CTAs, eight to two, with which all units fit 456.
@pytest.mark.parametrize("ctas,B", [(8, 14), (7, 15), (6, 18), (5, 21), (4, 27), (3, 36), (2, 55)])
@pytest.mark.parametrize("dt,i8", [("bf16", False), ("f16", True), ("f32", False)])
def test_clusters_of_every_size(ctas, B, dt, i8):
    """Lists from no tile to more than three a CTA, so that some parts are empty."""
    assert B * 4 * ctas <= 456 and (ctas == 8 or B * 4 * (ctas + 1) > 456)
    full = 64 * 3 * ctas + 17
    lens = [full] + [(0, 1, 63, 64, 65, 64 * ctas - 1, 64 * ctas, 64 * ctas + 1, full // 2)[b % 9] for b in range(1, B)]
    run(dt, 128, 16, 4, 16, lens, 30, i8=i8)


@pytest.mark.parametrize("dt,i8", [("bf16", False), ("f16", False), ("bf16", True), ("f32", False)])
def test_whole_units_and_shares(dt, i8):
    run(dt, 64, 16, 8, 16, [1 + 37 * b % 131 for b in range(60)], 10, i8=i8)
    run(dt, 64, 16, 8, 16, [1 + 577 * b % 1801 for b in range(60)], 30, i8=i8)
