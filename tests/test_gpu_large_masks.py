"""Large finite masks beside ordinary keys (padding of a prompt's start, whole key
tiles of it first), and masks whose float32 spacing is of the size of scores."""
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


def paged(q, k, v, mask, **kw):
    """decode_paged over the rows of contiguous k and v [B, G, n, D]; every way of dividing comes with the sizes."""
    B, G, n, D = k.shape
    pad = -n % 16
    pools = [torch.nn.functional.pad(t, (0, 0, 0, pad)).view(B, G, -1, 16, D).transpose(1, 2).reshape(-1, G, 16, D)
             for t in (k, v)]
    table = torch.arange(pools[0].shape[0], dtype=torch.int32, device="cuda").view(B, -1)
    o, lse = attn.decode_paged(q.transpose(1, 2), *pools, table, mask=mask, max_rows=n, return_lse=True, **kw)
    return o.transpose(1, 2), lse


def decode(q, k, v, mask, **kw):
    o, lse = attn.decode(q.transpose(1, 2), k, v, mask=mask, return_lse=True, **kw)
    return o.transpose(1, 2), lse


def forward(q, k, v, mask, **kw):
    return attn.fwd(q, k, v, layout="bhsd", mask=mask, return_lse=True, **kw)


def window(q, k, v, mask, **kw):
    n = k.shape[2]
    return attn.fwd(q, k, v, layout="bhsd", mask=mask, return_lse=True, causal=True, causal_offset=n, window_left=2 * n,
                    first_keys=3, **kw)


CALLS = dict(paged=paged, decode=decode, forward=forward, window=window)


@pytest.mark.parametrize("value", [-1e9, -3e4, -1.5e8, sb.LOW, -1e20])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("call,B,H,G,Sq,n,D", [
    ("forward", 2, 4, 2, 200, 700, 64), ("forward", 1, 2, 1, 130, 900, 128), ("forward", 2, 2, 1, 40, 600, 256),
    ("window", 2, 4, 2, 200, 700, 64), ("window", 1, 2, 1, 30, 900, 128), ("window", 2, 2, 1, 50, 300, 32),
    ("paged", 3, 8, 2, 1, 900, 128), ("paged", 60, 8, 8, 1, 90, 64), ("paged", 58, 8, 8, 1, 1800, 64),
    ("decode", 3, 8, 2, 1, 900, 128), ("decode", 2, 4, 2, 1, 2000, 64),
])
def test_padded_starts(call, B, H, G, Sq, n, D, dt, value):
    """Up to two thirds of the keys in front carry the value; rows of an entry's last pattern carry it throughout."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n + D)
    q, k, v = (torch.randn(B, h, m, D, generator=g, device="cuda").to(DT[dt]) for h, m in ((H, Sq), (G, n), (G, n)))
    pad = torch.randint(n // 4, 2 * n // 3, (B,), generator=g, device="cuda")
    mask = torch.where(torch.arange(n, device="cuda") < pad[:, None], value, 0.0)[:, None, None].contiguous()
    o, lse, tol, tol_l = sb.attention(q, k, v, torch.ones(B, Sq, n, dtype=torch.bool, device="cuda"),
                                      p="halves" if call == "paged" else "single", mask=mask)
    got, got_l = CALLS[call](q, k, v, mask)
    sb.check(got, o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")


@pytest.mark.parametrize("base,gap", [(-1.5e8, 16), (-1.5e8, 32), (-7e7, 8), (-2.0 ** 27, 16), (3e7, 4), (-5e5, 10)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("call,Sq,D,n", [("forward", 140, 64, 500), ("window", 140, 64, 500), ("window", 140, 128, 500),
                                         ("paged", 1, 64, 9000), ("paged", 1, 128, 77), ("window", 50, 32, 300)])
def test_spacing_of_masks(call, Sq, D, n, dt, base, gap):
    """A row masked with `base` throughout, where some keys' scores lie a step of its float32 spacing above: by that
    step and no more they outweigh the others, wherever the first of them comes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n + gap)
    q, k = (torch.zeros(1, 1, m, D, dtype=DT[dt], device="cuda") for m in (Sq, n))
    v = torch.randn(1, 1, n, D, generator=g, device="cuda").to(DT[dt])
    base = float(torch.tensor(base, dtype=torch.float32) // 64 * 64)   # on a multiple of every spacing here
    up = torch.rand(n, generator=g, device="cuda") < 0.02
    up[:n // 10] = False
    up[-2] = True
    q[..., 0] = 1
    k[0, 0, :, 0] = torch.where(up, float(gap), 0.0).to(DT[dt])
    x = torch.where(up, base + gap, base).double()
    assert torch.equal(x.float().double(), x)
    w = torch.softmax(x, 0)
    o = (w @ v[0, 0].double()).expand(1, 1, Sq, D)
    lse = torch.logsumexp(x, 0).expand(1, 1, Sq)
    rel = sb.p_error(DT[dt], "halves" if call == "paged" else "single")[0]
    tol = (rel + 2.0 ** -18) * (w @ v[0, 0].double().abs()) + sb.HALF[DT[dt]] * o.abs() + 2.0 ** -20
    got, got_l = CALLS[call](q, k, v, torch.full((1, 1, 1, n), base, device="cuda"), scale=1.0)
    sb.check(got, o, tol, "O")
    # (the logarithm of the sum is up to seven: under the spacing of the larger masks)
    assert float((got_l.double() - lse).abs().max()) <= max(abs(base) * 2.0 ** -23, 1e-4)
