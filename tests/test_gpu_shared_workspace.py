"""attn_fwd_shared writes and reads its workspace up to the size that the query gives, whatever the plan."""
from __future__ import annotations

import pytest

import shared_cases as sc
from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
GUARD = 1 << 22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


# dtype, D, B, Sq, H, G, page size, prefix rows, own lengths, options
CASES = [
    ("bf16", 128, 60, 1, 8, 2, 16, 4000, [1 + (7 * b) % 90 for b in range(60)], {}),   # packed, own keys whole units
    ("bf16", 128, 3, 1, 8, 2, 16, 60000, [9000, 1, 5000], {}),                         # ... cut, fragments behind the prefix's
    ("f16", 64, 70, 1, 8, 8, 16, 5000, [(7 * b) % 131 for b in range(70)], dict(max_rows=9000)),
    ("f16", 64, 80, 1, 8, 8, 16, 1000, [0] * 80, dict(max_rows=0)),                    # the prefix alone
    ("f16", 128, 30, 4, 8, 2, 16, 3000, [1 + (7 * b) % 90 for b in range(30)], {}),    # a few tokens, own items
    ("bf16", 64, 40, 3, 4, 4, 16, 5003, [(7 * b) % 90 for b in range(40)], dict(max_rows=4000)),   # ... in parts
    ("bf16", 128, 2, 73, 12, 4, 128, 20040, [55, 79], {}),                             # each entry by itself, lists cut
    ("f16", 64, 1, 471, 4, 1, 24, 119, [1420], {}),
    ("bf16", 128, 2, 805, 8, 4, 16, 3001, [800, 817], dict(offset=40)),
    ("f16", 128, 2, 301, 8, 2, 32, 5288, [453, 624], dict(causal=False)),
    ("bf16", 128, 4, 1, 8, 2, 16, 3000, [1, 30000, 37, 64], {}),                       # the decode pass alone, cut
    ("f32", 64, 70, 1, 8, 8, 7, 7003, [(3 * b) % 40 for b in range(70)], {}),          # float32: packed, own keys by decode
    ("f32", 128, 60, 1, 16, 4, 16, 6003, [1 + (5 * b) % 90 for b in range(59)] + [9000], {}),
    ("f32", 128, 20, 3, 8, 4, 16, 3001, [(5 * b) % 90 for b in range(20)], {}),        # ... own lists in parts
    ("f32", 64, 5, 33, 12, 4, 16, 501, [33, 40, 77, 100, 20], {}),                     # each entry in parts
    ("f32", 64, 3, 1, 12, 4, 16, 501, [33, 0, 20000], {}),
    ("f32", 256, 2, 9, 4, 2, 16, 700, [9, 12], {}),
    ("bf16", 256, 3, 1, 8, 2, 16, 500, [9, 20000, 0], {}),
    ("bf16", 80, 2, 12, 4, 2, 16, 700, [12, 70], {}),                                  # the CUDA cores
    ("bf16", 128, 2, 6, 8, 2, 16, 900, [6, 50], dict(i8="channel")),
    ("bf16", 128, 20, 7, 8, 2, 16, 4000, [9, 12] * 10, dict(pad=2)),                   # ... for rows off their boundaries
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_stays_inside_the_size_asked_for(i, monkeypatch):
    """The bytes on both sides of a workspace of the asked size stay as they were; what it holds before the call does
    not matter."""
    dt, D, B, Sq, H, G, ps, prefix, lens, opt = CASES[i]
    c = sc.make(dt, D, B, Sq, H, G, ps, prefix, lens, 600 + i, **opt)
    sizes, query = [], attn.attn_fwd_shared_workspace_size

    def recorded(*a):
        sizes.append(query(*a))
        return sizes[-1]

    monkeypatch.setattr(attn, "attn_fwd_shared_workspace_size", recorded)
    want, want_lse = sc.run(c, return_lse=True)
    n = sizes[-1]
    assert n > 0
    for fill in (255, 0):
        ws = torch.full((GUARD + n + GUARD,), fill, dtype=torch.uint8, device="cuda")
        out, lse = sc.run(c, return_lse=True, workspace=ws[GUARD:GUARD + n])
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert (ws[:GUARD] == fill).all() and (ws[GUARD + n:] == fill).all()
    with pytest.raises(attn.AttnError):
        sc.run(c, workspace=ws[GUARD:GUARD + n - 1])


@pytest.mark.parametrize("dt,Sq,B", [("bf16", 1, 60), ("f16", 4, 30), ("bf16", 150, 2), ("f32", 1, 70), ("f32", 20, 3)])
def test_a_scale_with_no_value_in_base_2(dt, Sq, B):
    """Scales whose product with log2(e) is infinite are taken too: queries of zero see the mean of V."""
    lens = [Sq + b % 20 for b in range(B)]
    c = sc.make(dt, 64, B, Sq, 8, 8, 16, 3000, lens, 700, scale=3e38)
    c["call"][0].zero_()
    out, lse = sc.run(c, return_lse=True)
    c["ref_kw"]["scale"] = 1.0
    sc.check(c, out, lse)
