"""Infinite and NaN values in V rows that a query sees: a positive weight times an
infinity is that infinity, both signs together and a NaN give NaN, and the other
columns, heads and entries are as they are without them."""
from __future__ import annotations

import math

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


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,H,G,lens,opt", [
    (128, 8, 2, [500, 37], {}),                             # clusters
    (64, 8, 8, [37 + i for i in range(60)], {}),            # whole units
    (64, 16, 8, [1500 + 7 * i for i in range(58)], {}),     # shares
    (256, 4, 2, [300, 5], {}),
    (128, 32, 2, [200, 90], dict(mask=True)),
    (128, 4, 2, [700, 300], dict(far=True)),                # infinities behind keys of small weight
    (128, 8, 2, [500, 200], dict(flat=True)),               # equal weights: probabilities of one
    (80, 4, 2, [100, 30], {}),
])
def test_paged_infinite_values(dt, D, H, G, lens, opt):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(lens) + D)
    B, ps, rows = len(lens), 16, max(lens)
    width = -(-rows // ps)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v = rand(B, 1, H, D).to(DT[dt]), rand(B * width, G, ps, D).to(DT[dt]), rand(B * width, G, ps, D).to(DT[dt])
    if opt.get("flat"):
        k.zero_()
    if opt.get("far"):      # the infinities' keys 14 nats below: 2^-20
        q, k = q.zero_(), k.zero_()
        q[..., 0], k[..., 0] = 1, 14
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, m in enumerate(lens):
        for col, r, x in ((1, 0, math.inf), (2, m - 1, -math.inf), (3, m // 2, math.inf), (3, m // 3, -math.inf),
                          (5, m // 2, math.nan), (D - 1, m // 4, math.inf), (D - 2, m // 5, -math.inf)):
            page = b * width + r // ps
            v[page, b % G, r % ps, col] = x
            if opt.get("far"):
                k[page, :, r % ps, 0] = 0
    mask = rand(B, 1, 1, rows) if opt.get("mask") else None
    vis = (torch.arange(rows, device="cuda")[None] < n[:, None])[:, None]
    o, lse, tol, tol_l = sb.attention(q.transpose(1, 2), sb.rows_of(k, table, ps, rows), sb.rows_of(v, table, ps, rows),
                                      vis, mask=mask, scale=1.0 if opt.get("far") else 0.0)
    assert (o == math.inf).any() and (o == -math.inf).any() and torch.isnan(o).any()
    got, got_l = attn.decode_paged(q, k, v, table, n, mask=mask, max_rows=rows, return_lse=True,
                                   scale=1.0 if opt.get("far") else 0.0)
    sb.check(got.transpose(1, 2), o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")
