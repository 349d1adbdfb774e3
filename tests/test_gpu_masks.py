"""Additive masks of any size in attn_fwd, attn_decode and attn_decode_append: values down to float32's lowest hide
nothing by themselves, and large ones that a whole row carries leave it the mean of their keys."""
from __future__ import annotations

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


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,B,H,G,Sq,Sk,opt", [
    (128, 1, 4, 2, 300, 500, {}),
    (64, 2, 4, 4, 270, 300, dict(sink=True)),
    (128, 3, 2, 1, 200, 400, dict(bcast=True)),               # a staged mask: rows of an entry alike
    (64, 8, 4, 2, 100, 700, dict(bcast=True, causal=True)),   # paired heads
    (256, 1, 2, 1, 300, 400, {}),
    (256, 8, 2, 2, 150, 300, dict(bcast=True)),
    (128, 1, 2, 2, 200, 300, dict(softcap=20.0)),
    (64, 1, 2, 2, 200, 300, dict(scale=-0.1)),
    (256, 1, 2, 2, 150, 300, dict(softcap=20.0, sink=True)),
    (128, 1, 2, 1, 90, 1200, dict(splits=5)),
    (64, 1, 2, 1, 90, 1100, dict(splits=3, sink=True, causal=True)),
    (256, 1, 2, 1, 90, 1000, dict(splits=4)),
    (96, 1, 2, 1, 60, 300, {}),
])
def test_forward(dt, D, B, H, G, Sq, Sk, opt):
    forward(dt, D, B, H, G, Sq, Sk, opt)


@pytest.mark.parametrize("D,B,H,G,Sq,Sk,opt", [
    (64, 1, 2, 1, 100, 300, {}), (128, 1, 2, 2, 60, 2500, dict(sink=True)), (80, 1, 2, 2, 50, 900, dict(splits=4)),
])
def test_forward_f32(D, B, H, G, Sq, Sk, opt):
    forward("f32", D, B, H, G, Sq, Sk, opt)


def forward(dt, D, B, H, G, Sq, Sk, opt):
    g = gen(D + Sq + Sk)
    q, k, v = (randn(g, B, h, n, D, dt=DT[dt]) for h, n in ((H, Sq), (G, Sk), (G, Sk)))
    mask = sb.mask_kinds(g, B, 1, 1 if opt.get("bcast") else Sq, Sk)
    sink = randn(g, H) if opt.get("sink") else None
    lens = torch.randint(Sk // 2, Sk + 1, (B,), generator=g, device="cuda").to(torch.int32)
    vis = (torch.arange(Sk, device="cuda") < lens[:, None])[:, None].expand(B, Sq, Sk)
    if opt.get("causal"):
        vis = vis & (torch.arange(Sk, device="cuda") <= torch.arange(Sq, device="cuda")[:, None] + Sk - Sq)
    kw = dict(scale=opt.get("scale", 0.0), softcap=opt.get("softcap", 0.0))
    o, lse, tol, tol_l = sb.attention(q, k, v, vis, p="single", mask=mask, sink=sink, **kw)
    got, got_l = attn.fwd(q, k, v, layout="bhsd", mask=mask, head_sink=sink, masked_rows="zero", return_lse=True,
                          key_splits=opt.get("splits", 0), k_lens=lens, causal=opt.get("causal", False), **kw)
    sb.check(got, o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")


@pytest.mark.parametrize("dt,D,H,G,cap,opt", [
    ("bf16", 128, 8, 2, 900, {}), ("f16", 128, 8, 8, 3000, dict(sink=True)), ("bf16", 128, 20, 1, 700, dict(softcap=9.0)),
    ("bf16", 128, 8, 2, 900, dict(i8=True)), ("f16", 128, 16, 2, 2000, dict(i8=True, softcap=9.0)),
    ("f16", 64, 4, 2, 700, {}), ("f32", 128, 4, 2, 700, {}), ("f32", 64, 4, 2, 700, dict(sink=True)),
])
def test_decode(dt, D, H, G, cap, opt):
    g, B = gen(D + H + cap), 24
    i8 = opt.get("i8")
    if i8:
        k, v = (torch.randint(-128, 128, (B, G, cap, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
        sc = [torch.rand(G * D, generator=g, device="cuda") * 0.015 + 0.005 for _ in range(2)]
    else:
        k, v, sc = randn(g, B, G, cap, D, dt=DT[dt]), randn(g, B, G, cap, D, dt=DT[dt]), None
    q = randn(g, B, 1, H, D, dt=DT[dt])
    n = torch.randint(1, cap + 1, (B,), generator=g, device="cuda").to(torch.int32)
    mask = sb.mask_kinds(g, B, 1, 1, cap)
    sink = randn(g, H) if opt.get("sink") else None
    vis = (torch.arange(cap, device="cuda") < n[:, None])[:, None]
    # an int8 cache's pass rounds the scaled query and P to f16, and biases its integers by 1152 of 127 at most
    o, lse, tol, tol_l = sb.attention(q.transpose(1, 2), k, v, vis, p="single", mask=mask, sink=sink, kv_scales=sc,
                                      softcap=opt.get("softcap", 0.0), extra_score=2.0 ** -11 if i8 else 0.0)
    if i8:
        top = torch.where(vis.transpose(1, 2)[:, None], v.double() * sc[1].double().view(1, G, 1, D), 0.0).abs().amax((2, 3))
        tol = tol + 11 * 2.0 ** -11 * top.repeat_interleave(H // G, 1)[:, :, None, None]
        tol_l = tol_l + 2.0 ** -10
    kw = dict(k_scale=sc[0], v_scale=sc[1]) if i8 else {}
    got, got_l = attn.decode(q, k, v, n, mask=mask, head_sink=sink, softcap=opt.get("softcap", 0.0), masked_rows="zero",
                             return_lse=True, **kw)
    sb.check(got.transpose(1, 2), o, tol, "O")
    sb.check(got_l, lse, tol_l, "LSE")
    assert sink is not None or (lse == sb.LOW).any()
