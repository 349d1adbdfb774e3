"""attn_fwd_shared: a visible key whose score is NaN makes its row NaN in O and
LSE, also where a part of the keys has no other score, however the keys are
cut into parts; and no other row."""
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


# dtype, D, B, Sq, H, G, page size, prefix rows, own lengths, options
CASES = [
    ("bf16", 128, 60, 1, 8, 2, 16, 4000, [1 + (7 * b) % 90 for b in range(60)], {}),      # many parts of few rows
    ("f16", 64, 150, 1, 8, 8, 16, 3001, [1 + (7 * b) % 90 for b in range(150)], {}),      # ... of more
    ("bf16", 128, 40, 1, 8, 8, 16, 1000, [1 + b % 20 for b in range(40)], {}),            # few parts
    ("f16", 64, 80, 1, 8, 8, 16, 1000, [1 + b % 20 for b in range(80)], {}),
    ("bf16", 128, 3, 1, 8, 2, 16, 60000, [9000, 1, 5000], {}),                            # own keys cut among CTAs
    ("f16", 128, 30, 4, 8, 2, 16, 3000, [1 + (7 * b) % 90 for b in range(30)], {}),       # a few tokens, packed
    ("bf16", 64, 40, 3, 4, 4, 16, 5003, [1 + (7 * b) % 90 for b in range(40)], {}),
    ("bf16", 128, 2, 73, 12, 4, 128, 20040, [55, 79], {}),                                # units cut 19, 8, 7 and 4 times
    ("f16", 128, 2, 301, 8, 2, 32, 5288, [453, 624], {}),
    ("f16", 64, 1, 471, 4, 1, 24, 119, [1420], {}),
    ("bf16", 128, 2, 805, 8, 4, 16, 3001, [800, 817], {}),
    ("bf16", 128, 4, 1, 8, 2, 16, 300, [1, 100, 37, 64], {}),                             # the decode pass alone
    ("f32", 64, 70, 1, 8, 8, 7, 7003, [1 + (3 * b) % 40 for b in range(70)], {}),         # float32: packed, own keys by it
    ("f32", 128, 20, 3, 8, 4, 16, 3001, [1 + (5 * b) % 90 for b in range(20)], {}),       # ... in parts
    ("f32", 64, 5, 33, 12, 4, 16, 501, [33, 40, 77, 100, 20], {}),                        # each entry in parts
    ("f32", 64, 3, 1, 12, 4, 16, 501, [33, 1, 100], {}),
    ("f32", 256, 2, 9, 4, 2, 16, 700, [9, 12], {}),
    ("bf16", 80, 2, 12, 4, 2, 16, 700, [12, 70], {}),                                     # the CUDA cores
    ("bf16", 128, 3, 1, 8, 2, 16, 400, [1, 50, 3], dict(i8="channel")),
]


def options(H, sink):
    return dict(masked_rows="zero", head_sink=torch.linspace(-3.0, 8.0, H, device="cuda") if sink else None)


def check(c, bad, i8=False):
    """bad [B, H, Sq]: the rows that have to be NaN."""
    out, lse = sc.run(c, return_lse=True)
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(out).all(-1).transpose(1, 2), bad)
    sc.check(c, out, lse, **(dict(extra_score=2.0 ** -22) if i8 else {}))


def some_rows(B, H, Sq):
    """Rows here and there, more than one of an entry and of a head."""
    n = B * H * Sq
    at = torch.arange(n, device="cuda")
    return ((at * 7 + 3) % 11 == 0).view(B, H, Sq)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_queries(i, sink):
    """A NaN in a query: every score of the row is NaN, in every part."""
    dt, D, B, Sq, H, G, ps, prefix, lens, opt = CASES[i]
    c = sc.make(dt, D, B, Sq, H, G, ps, prefix, lens, 300 + i, **options(H, sink), **opt)
    bad = some_rows(B, H, Sq)
    c["call"][0][bad.transpose(1, 2), 5] = math.nan
    check(c, bad, "i8" in opt)


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_masks(i, sink):
    """Rows with one NaN among -inf: alone in the row, in front of finite scores, behind them, in their middle."""
    dt, D, B, Sq, H, G, ps, prefix, lens, opt = CASES[i]
    keys = prefix + max(lens)
    mask = torch.zeros(B, H, Sq, keys, device="cuda")
    bad = some_rows(B, H, Sq)
    c = sc.make(dt, D, B, Sq, H, G, ps, prefix, lens, 400 + i, mask=mask, **options(H, sink), **opt)
    vis = c["ref"][3]
    for n, (b, h, q) in enumerate(bad.nonzero().tolist()):
        row, last = mask[b, h, q], int(vis[b, q].nonzero().max())   # (its last visible key)
        if n % 5 == 0:
            row[:], row[(n * 61) % prefix] = -math.inf, math.nan
        elif n % 5 == 1:
            row[:prefix], row[(n * 37) % prefix] = -math.inf, math.nan
        elif n % 5 == 2:
            row[prefix:], row[last] = -math.inf, math.nan
        elif n % 5 == 3:
            at = (n * 53) % prefix
            row[max(at - 2500, 0):at + 2500], row[at] = -math.inf, math.nan
        else:
            row[:], row[last] = -math.inf, math.nan
    # Rows with nothing but -inf next to them are masked rows, no NaN rows.
    gone = some_rows(B, H, Sq).roll(1, 0) & ~bad if B > 1 else torch.zeros_like(bad)
    mask[gone] = -math.inf
    check(c, bad, "i8" in opt)


@pytest.mark.parametrize("i", [i for i, c in enumerate(CASES) if c[3] == 1 and "i8" not in c[9]])
def test_first_own_key(i):
    """The first token of an entry, whose only own key holds a NaN: its rows are NaN."""
    dt, D, B, Sq, H, G, ps, prefix, lens, opt = CASES[i]
    c = sc.make(dt, D, B, Sq, H, G, ps, prefix, lens, 500 + i, **options(H, False), **opt)
    q, k, v, ptab, _, table = c["call"]
    bad = torch.zeros(B, H, Sq, dtype=torch.bool, device="cuda")
    for b in (b for b in range(B) if lens[b] == 1):
        k[table[b, 0].long(), 0, 0, 3] = math.nan
        c["ref"][1][b, 0, prefix, 3] = math.nan
        bad[b, :H // G] = True
    assert bad.any()
    check(c, bad)
