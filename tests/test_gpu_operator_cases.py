"""The measured cases of the serving operators (perf/operators.py), their largest
shapes among them, through the library once: element by element against float64
under bounds that follow each row, and the quick ones against the file's own
64-bit definition too."""
from __future__ import annotations

import importlib.util
import os
import random

import pytest

import serving_bounds as sb
from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
QUICK = 2e9   # multiply-adds up to which the file's own definition takes a moment


def load():
    spec = importlib.util.spec_from_file_location("operator_cases", os.path.join(ROOT, "perf", "operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


OPS = load()
rng = random.Random(5)
CASES = OPS.listed() + [dict(OPS.draw(rng), name=f"drawn{i}") for i in range(6)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


def paged(c, s, got):
    for b, n in enumerate(OPS._lens(c)):
        if n == 0:
            assert (got["o"][b] == 0).all()
            continue
        j = torch.arange(n, device="cuda")
        vis = (j >= 0) if c["window"] < 0 else (j >= n - 1 - c["window"]) | (j < c["first"])
        table = s["table"][b:b + 1].clamp(min=0)   # (pages behind the window are not in the list)
        k, v = (sb.rows_of(s[x], table, c["ps"], n, c["nhd"]) for x in "kv")
        o, _, tol, _ = sb.attention(s["q"][b:b + 1].transpose(1, 2), k, v, vis[None, None],
                                    kv_scales=(s["ks"], s["vs"]) if "ks" in s else None,
                                    extra_score=2.0 ** -22 if "ks" in s else 0.0)
        sb.check(got["o"][b:b + 1].transpose(1, 2), o, tol, f"entry {b}")


def window(c, s, got):
    q, k, v, o = (t.transpose(1, 2) if c["bshd"] else t for t in (s["q"], s["k"], s["v"], got["o"]))
    per = c["H"] // c["G"]
    j = torch.arange(c["k_len"], device="cuda")
    for b, n in enumerate(OPS._lens(c)):
        diag = (torch.arange(c["q_len"], device="cuda") + n - c["q_len"])[:, None]
        start = s["seg"][b][:, None] if c["docs"] else torch.zeros_like(diag)
        vis = (j < n) & (j <= diag) & (j >= start) & ((j >= diag - c["window"]) | (j < start + c["first"]))
        for g in range(c["G"]):
            h = slice(g * per, (g + 1) * per)
            want, _, tol, _ = sb.attention(q[b:b + 1, h], k[b:b + 1, g:g + 1], v[b:b + 1, g:g + 1], vis[None], p="single")
            sb.check(o[b:b + 1, h], want, tol, f"entry {b}, kv head {g}")


def prep(c, s, got, seed):
    want = OPS.exact(c, seed)
    D = c["D"]
    for name in "qkv":
        y = want[name]
        # a rotated element is two products of normed ones: as large as the row's largest, twice at most
        tol = (D / 2 + 11) * sb.U32 * 2 * y.abs().amax(-1, keepdim=True) + sb.HALF[OPS.DTYPES[c["dtype"]]] * y.abs()
        sb.check(got[name], y, tol + 2.0 ** -25, name)


@pytest.mark.parametrize("i", range(len(CASES)), ids=[c["name"] for c in CASES])
def test_case(i):
    c, seed = CASES[i], 100 + i
    OPS.own = True
    try:
        s = OPS.prepare(c, seed)
        got = {k: v.clone() for k, v in OPS.run(s).items()}
        again = OPS.run(s)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], again[k]) for k in got)
        assert attn.attn_device_status() == attn.ATTN_OK
        OPS.own = False
        if c["op"] == "prep":
            prep(c, s, got, seed)
            return
        (paged if c["op"] == "paged" else window)(c, s, got)
        if OPS.work(c)["flops"] < QUICK:
            want = OPS.exact(c, seed)["o"]
            plain = OPS.run(s)["o"]
            # the definition against the formula: rounded once, the plain form is as far off as the type's half step
            half = sb.HALF[OPS.DTYPES[c["dtype"]]]
            assert float((plain.double() - want).abs().max()) <= 1.01 * half * float(want.abs().max()) + 2.0 ** -16
            assert float((got["o"].double() - want).abs().max()) <= 4 * half * float(want.abs().max()) + 2.0 ** -16
    finally:
        OPS.own = False
