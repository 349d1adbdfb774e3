"""Long rows whose weight is spread over keys far below the largest: every key
counts, also where f16 alone could not hold its probability."""
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


# One key lies `below` log2 units above n others, which share one score.  With e = 2^-below, a column of V that is 1
# for the others and 0 for the one gives n e / (1 + n e): its sum holds the small weights alone.  A column of ones
# gives 1; there every product joins a float32 sum of 1, and of those under 2^-24 of it none may be left.


def expected(n, e):
    """O of the columns (ones; ones for the others) for n others (a tensor) of weight e, and LSE less the first score."""
    den = 1 + n * e
    return torch.stack([torch.ones_like(den), 1 - 1 / den], -1), torch.log(den)


def bounds(dt, how, n, o, ds):
    """O: the row sum takes n / 32 float32 steps a lane at least, the second column as many of its own; what a
    probability loses (serving_bounds.py); ds, the score's error; the output's rounding.  First column: the products
    that a sum of 1 absorbs, and LSE."""
    rel, floor = sb.p_error(dt, how)
    sums = (16 + n / 32) * sb.U32
    own = o[..., 1:] * (2 * sums + rel + 2 * ds + 2.0 ** -20 + sb.HALF[dt]) + 2 * floor * n
    return torch.cat([own * 0 + 2 * n * sb.U32 + sums + rel + sb.HALF[dt], own], -1), sums + 2 * ds + 2.0 ** -18


@pytest.mark.parametrize("dt,i8", [("f16", False), ("bf16", False), ("f32", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("below", [20, 25.2, 31])
@pytest.mark.parametrize("at", [0, 700000])
def test_paged_spread_weight(dt, i8, below, at):
    """Entries enough that a CTA walks long lists alone: 2^21 rows each, all pages but one the same page."""
    n, D, ps, B = 2 ** 21, 64, 128, 500
    q = torch.zeros(B, 1, 1, D, device="cuda", dtype=DT[dt])
    q[..., 0] = 1
    score = torch.tensor(below * math.log(2)).to(DT[dt])
    k = torch.zeros(2, 1, ps, D, device="cuda", dtype=torch.int8 if i8 else DT[dt])
    v = torch.ones_like(k)
    k[1, 0, 5, 0] = 127 if i8 else score
    v[1, 0, 5, 1] = 0
    table = torch.zeros(B, n // ps, dtype=torch.int32, device="cuda")
    table[:, at // ps] = 1
    kw = dict(k_scale=score.float().view(1).cuda() / 127, v_scale=torch.ones(1, device="cuda")) if i8 else {}
    got, lse = attn.decode_paged(q, k, v, table, scale=1.0, return_lse=True, **kw)
    top = float(kw["k_scale"].double() * 127) if i8 else float(score.double())
    others, e = torch.tensor(n - 1.0, dtype=torch.float64, device="cuda"), math.exp(-top)
    o, l = expected(others, e)
    tol, tol_l = bounds(DT[dt], "halves", n, o, top * 2.0 ** -20)
    assert float(((got[:, 0, 0, :2].double() - o).abs() / tol).max()) <= 1
    assert float((lse[:, 0, 0].double() - (l + top)).abs().max()) <= tol_l


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("below", [20, 25.2, 28])
@pytest.mark.parametrize("D,mask", [(64, False), (128, True)])
def test_window_spread_weight(dt, below, D, mask):
    """Query blocks enough that a block's list is one CTA's, and a window of up to 2^17 keys."""
    n, Sq, w = 2 ** 17, 20480, 130000
    q = torch.zeros(1, 1, Sq, D, device="cuda", dtype=DT[dt])
    k = torch.zeros(1, 1, n, D, device="cuda", dtype=DT[dt])
    q[..., 0] = 1
    k[0, 0, 0, 0] = below * math.log(2)
    v = torch.ones_like(k)
    v[0, 0, 0, 1] = 0
    got, lse = attn.fwd(q, k, v, layout="bhsd", causal=True, window_left=w, first_keys=3, scale=1.0, return_lse=True,
                        mask=torch.zeros(1, 1, 1, n, device="cuda") if mask else None)
    top = float(k[0, 0, 0, 0].double())
    diag = torch.arange(Sq, device="cuda", dtype=torch.float64) + n - Sq
    near = (diag - w).clamp(min=0)
    others = diag + 1 - near + near.clamp(max=3) - 1
    o, l = expected(others, math.exp(-top))
    tol, tol_l = bounds(DT[dt], "single", n, o, top * 2.0 ** -20)
    assert float(((got[0, 0, :, :2].double() - o).abs() / tol).max()) <= 1
    assert float((lse[0, 0].double() - (l + top)).abs().max()) <= tol_l
