"""The measured cases of perf/more_operators.py, their largest shapes among them,
through the library twice: the same bits, element by element against float64
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
    spec = importlib.util.spec_from_file_location("more_operator_cases", os.path.join(ROOT, "perf", "more_operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


OPS = load()
rng = random.Random(11)
CASES = OPS.listed() + [dict(OPS.draw(rng), name=f"drawn{i}") for i in range(10)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


def shared(c, s, got):
    per, P, q = c["H"] // c["G"], c["prefix"], c["q"]
    pre = [sb.rows_of(s[x], s["prefix"][None], c["ps"], P, c["nhd"]) for x in "kv"]
    for b, n in enumerate(OPS._lens(c)):
        if b % max(1, c["B"] // 6):
            continue   # some entries of many
        own = [sb.rows_of(s[x], s["table"][b:b + 1], c["ps"], n, c["nhd"]) for x in "kv"]
        k, v = (torch.cat([p, o], 2) for p, o in zip(pre, own))
        step = max(1, int(2 ** 28 / (c["H"] * (P + n))))   # rows of a time's scores
        for i0 in range(0, q, step):
            i = torch.arange(i0, min(i0 + step, q), device="cuda")
            vis = torch.arange(P + n, device="cuda") - P <= (i + n - q)[:, None]
            vis[:, :P] = True
            for g in range(c["G"]):
                h = slice(g * per, (g + 1) * per)
                want, _, tol, _ = sb.attention(s["q"][b:b + 1, i][:, :, h].transpose(1, 2), k[:, g:g + 1], v[:, g:g + 1],
                                               vis[None], p="single")
                sb.check(got["o"][b:b + 1, i][:, :, h].transpose(1, 2), want, tol, f"entry {b}, kv head {g}, row {i0}")


def axes(c, got, seed):
    want = OPS.exact(c, seed)
    for name in "qkv":
        y = want[name]
        # a rotated element is two products of normed ones: as large as the row's largest, twice at most
        tol = (c["D"] / 2 + 11) * sb.U32 * 2 * y.abs().amax(-1, keepdim=True) + sb.HALF[OPS.DTYPES[c["dtype"]]] * y.abs()
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
        if c["op"] == "axes":
            axes(c, got, seed)
            return
        shared(c, s, got)
        if OPS.work(c)["flops"] < QUICK:
            want = OPS.exact(c, seed)["o"]
            plain = OPS.run(s)["o"]
            half = sb.HALF[OPS.DTYPES[c["dtype"]]]
            # rounded once, the plain form is as far off as the type's half step, beside float32's own sums
            assert float((plain.double() - want).abs().max()) <= 1.01 * half * float(want.abs().max()) + 2.0 ** -16
            assert float((got["o"].double() - want).abs().max()) <= 4 * half * float(want.abs().max()) + 2.0 ** -16
    finally:
        OPS.own = False
