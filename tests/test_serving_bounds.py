"""The bounds of serving_bounds.py against planted mistakes, on the CPU: a lost key
tile, a stale one or a wrong row is beyond them in lists of any length, and a
float32 evaluation of the formula is within them."""
from __future__ import annotations

import pytest

import serving_bounds as sb

torch = pytest.importorskip("torch")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def case(dt, n, D, H, G, seed=1, marked=64):
    """One entry's list in which `marked` keys, spread from its first to its last row, hold most of the weight: what
    a tile of any place adds to the result does not shrink with the list."""
    g = torch.Generator()
    g.manual_seed(seed)
    q, k, v = (torch.randn(1, h, m, D, generator=g).to(DT[dt]) for h, m in ((H, 1), (G, n), (G, n)))
    at = torch.linspace(0, n - 1, marked).long()
    u = q.view(G, H // G, D)[:, 0].float()
    u = u / u.norm(dim=-1, keepdim=True)
    k[0, :, at] = (k[0, :, at].float() + 25 * u[:, None]).to(DT[dt])
    return q, k, v, at


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [200, 9000, 100003])
def test_bounds_hold_and_reject(dt, n):
    q, k, v, at = case(dt, n, 64, 2, 2)
    vis = torch.ones(1, 1, n, dtype=torch.bool)
    o, lse, tol, tol_l = sb.attention(q, k, v, vis)
    # the formula in float32, rounded once
    x = q.float() @ k.float().transpose(-1, -2) * 64 ** -0.5
    p = torch.exp(x - x.amax(-1, keepdim=True))
    plain = (p @ v.float() / p.sum(-1, keepdim=True)).to(DT[dt])
    assert sb.worst(plain, o, tol) <= 1
    assert sb.worst(x.logsumexp(-1), lse, tol_l) <= 1
    # mistakes in V, in K, and in which rows are read, tile by tile
    w = torch.softmax((q.double() @ k.double().transpose(-1, -2)) * 64 ** -0.5, -1)
    for first in {0, int(at[len(at) // 2]) // 16 * 16, (n - 1) // 16 * 16}:
        tile = slice(first, min(first + 16, n))
        lost = v.double().clone()
        lost[:, :, tile] = 0
        assert sb.worst((w @ lost).to(DT[dt]), o, tol) > 1, "a tile of V that is zero"
        stale = v.double().clone()
        stale[:, :, tile] = v.double()[:, :, tile].roll(3, 2)
        if (tile.stop - tile.start) % 3:
            assert sb.worst((w @ stale).to(DT[dt]), o, tol) > 1, "rows of a tile in another order"
        kk = k.double().clone()
        kk[:, :, tile] = 0
        w2 = torch.softmax((q.double() @ kk.transpose(-1, -2)) * 64 ** -0.5, -1)
        assert sb.worst((w2 @ v.double()).to(DT[dt]), o, tol) > 1, "a tile of K that is zero"
    half = v.double().clone()
    half[:, 1] = v.double()[:, 0]
    assert sb.worst((w @ half).to(DT[dt]), o, tol) > 1, "another head's values"


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_ordinary_lists_reject_a_zeroed_tile(dt):
    """Without lifted keys too, at the longest ordinary list of the tests."""
    g = torch.Generator()
    g.manual_seed(3)
    n, D = 9000, 128
    q, k, v = (torch.randn(1, h, m, D, generator=g).to(DT[dt]) for h, m in ((8, 1), (2, n), (2, n)))
    o, _, tol, _ = sb.attention(q, k, v, torch.ones(1, 1, n, dtype=torch.bool))
    w = torch.softmax(q.double() @ k.double().repeat_interleave(4, 1).transpose(-1, -2) * D ** -0.5, -1)
    v2 = v.double().repeat_interleave(4, 1)
    v2[:, :, 4096:4160] = 0
    assert sb.worst((w @ v2).to(DT[dt]), o, tol) > 1
