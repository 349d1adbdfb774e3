"""Paged decode over int8 caches with large scores: a scaled query keeps its bits
(half a step of f16 in an element of a score of 200 would be 0.05 in the exponent)."""
from __future__ import annotations

import pytest

import serving_bounds as sb
from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,H,G,lens,size", [
    (128, 8, 2, [500, 37], 1.0),
    (128, 8, 2, [900, 300], 200.0),                          # one channel carries the score
    (64, 16, 1, [700, 333], 100.0),
    (256, 4, 2, [300, 50], 150.0),
    (64, 8, 8, [40 + i for i in range(60)], 120.0),          # whole units
    (128, 16, 8, [1500 + 3 * i for i in range(58)], 180.0),  # shares
])
def test_paged_int8_large_scores(dt, D, H, G, lens, size):
    g = torch.Generator(device="cuda")
    g.manual_seed(D + len(lens))
    B, ps, rows = len(lens), 16, max(lens)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(DT[dt])
    q[..., 3] = (size * (1 + 0.3 * torch.rand(B, 1, H, generator=g, device="cuda"))).to(DT[dt])
    k, v = (torch.randint(-128, 128, (80, G, ps, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    k[..., 3] = torch.randint(100, 128, (80, G, ps), generator=g, device="cuda", dtype=torch.int8)
    ks, vs = (torch.rand(G * D, generator=g, device="cuda") * 0.015 + 0.005 for _ in range(2))
    ks.view(G, D)[:, 3] = 0.0079
    table = torch.randint(0, 80, (B, -(-rows // ps)), generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    vis = (torch.arange(rows, device="cuda")[None] < n[:, None])[:, None]
    o, lse, tol, tol_l = sb.attention(q.transpose(1, 2), sb.rows_of(k, table, ps, rows), sb.rows_of(v, table, ps, rows),
                                      vis, kv_scales=(ks, vs), scale=1.0 if size > 1 else 0.0, extra_score=2.0 ** -22)
    got, got_l = attn.decode_paged(q, k, v, table, n, k_scale=ks, v_scale=vs, max_rows=rows, return_lse=True,
                                   scale=1.0 if size > 1 else 0.0)
    sb.check(got.transpose(1, 2), o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")
