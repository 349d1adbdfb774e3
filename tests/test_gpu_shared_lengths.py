"""attn_fwd_shared: no keys at all, lengths that are not given, last indices, lengths outside the room, padding entries."""
from __future__ import annotations

import math

import pytest

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


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("f32", 64), ("bf16", 80), ("f32", 256)])
@pytest.mark.parametrize("Sq", [1, 40])
def test_no_keys(dt, D, Sq):
    """No prefix and no room for own keys: masked rows, or the sink alone."""
    B, H = 3, 4
    c = sc.make(dt, D, B, Sq, H, 2, 16, 0, [0] * B, 1)
    sink = torch.linspace(-2.0, 3.0, H, device="cuda")
    for kw, value, lse_of in ((dict(masked_rows="nan"), math.nan, None), (dict(masked_rows="zero"), 0.0, None),
                              (dict(masked_rows="nan", head_sink=sink), 0.0, sink)):
        out, lse = sc.run(c, return_lse=True, **kw)
        assert torch.equal(torch.isnan(out), torch.full_like(out, value).isnan())
        assert (torch.nan_to_num(out) == 0).all()
        want = torch.full((B, H, Sq), -math.inf, device="cuda") if lse_of is None else lse_of.view(1, H, 1).expand(B, H, Sq)
        assert torch.allclose(lse, want, rtol=2.0 ** -22, atol=0) if lse_of is not None else torch.equal(lse, want)


@pytest.mark.parametrize("dt,D,B,Sq,H,G,prefix,room", [
    ("bf16", 128, 60, 1, 8, 2, 4000, 70), ("f16", 64, 80, 1, 8, 8, 1000, 20), ("f16", 128, 30, 4, 8, 2, 3000, 90),
    ("bf16", 128, 2, 301, 8, 2, 5288, 624), ("f32", 64, 70, 1, 8, 8, 7003, 40), ("f32", 64, 5, 33, 12, 4, 501, 100),
    ("bf16", 128, 4, 1, 8, 2, 300, 100), ("bf16", 80, 2, 12, 4, 2, 700, 70)])
def test_lengths(dt, D, B, Sq, H, G, prefix, room):
    """Without lengths an entry has its whole room; a last index is a length less one; lengths are cut to the room; an
    entry of padding (length 0, a list without pages) sees the prefix alone and no one sees it."""
    whole = sc.make(dt, D, B, Sq, H, G, 16, prefix, [room] * B, 2)
    out, lse = sc.run(whole, return_lse=True)
    sc.check(whole, out, lse)
    for lens in (None, whole["args"]["k_lens"] * 1000, torch.full_like(whole["args"]["k_lens"], 2 ** 31 - 1)):
        assert torch.equal(sc.run(whole, k_lens=lens), out)
    own = [(7 * b) % (room + 1) for b in range(B)]
    own[0] = 0
    c = sc.make(dt, D, B, Sq, H, G, 16, prefix, own, 3, max_rows=room)
    out, lse = sc.run(c, return_lse=True)
    sc.check(c, out, lse)
    n = c["args"]["k_lens"]
    assert torch.equal(sc.run(c, k_lens=n - 1, k_lens_kind="last_index"), out)
    assert torch.equal(sc.run(c, k_lens=torch.where(n == 0, -2 ** 31, n)), out)
    table = c["call"][5]
    table[0] = -1
    assert torch.equal(sc.run(c), out)
