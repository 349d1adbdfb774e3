"""The torch entry points of the serving operators refuse tensors whose extents,
types or devices the kernels would read or write past.  Extents are checked
before devices, so those refusals are shown with host tensors; the rest on a GPU."""
from __future__ import annotations

import pytest

from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
B, H, G, D, PS = 2, 4, 2, 64, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    attn.lib()


def paged(dev="cpu", i8=False):
    f16 = dict(device=dev, dtype=torch.float16)
    pool = torch.zeros(8, G, PS, D, device=dev, dtype=torch.int8 if i8 else torch.float16)
    kw = dict(q=torch.zeros(B, 1, H, D, **f16), k_pool=pool, v_pool=pool.clone(),
              table=torch.zeros(B, 4, dtype=torch.int32, device=dev),
              k_lens=torch.ones(B, dtype=torch.int32, device=dev))
    return dict(kw, k_scale=torch.ones(1, device=dev), v_scale=torch.ones(1, device=dev)) if i8 else kw


def prep(dev="cpu", i8=True):
    f16 = dict(device=dev, dtype=torch.float16)
    k = torch.zeros(B, 1, G, D, **f16)
    kc = torch.zeros(B, G, PS, D, device=dev, dtype=torch.int8 if i8 else torch.float16)
    kw = dict(q=torch.zeros(B, 1, H, D, **f16), k=k, v=k.clone(), k_cache=kc, v_cache=kc.clone())
    return dict(kw, k_scale=torch.ones(1, device=dev), v_scale=torch.ones(1, device=dev)) if i8 else kw


def window(dev="cpu"):
    f16 = dict(device=dev, dtype=torch.float16)
    kv = torch.zeros(B, G, 30, D, **f16)
    return dict(q=torch.zeros(B, H, 8, D, **f16), k=kv, v=kv.clone(), layout="bhsd", causal=True, window_left=9,
                first_keys=2)


SCALES = [(torch.ones(D), torch.ones(D)), (torch.ones(G * D), torch.ones(1)), (torch.ones(1), torch.ones(G * D)),
          (torch.ones(G * D), torch.ones(G * D - 1)), (torch.ones(2 * G * D)[::2], torch.ones(G * D)), (None, torch.ones(1)),
          (torch.ones(1), None)]


@pytest.mark.parametrize("i", range(len(SCALES)))
@pytest.mark.parametrize("call", [lambda **k: attn.decode_paged(**dict(paged(i8=True), **k)),
                                  lambda **k: attn.qkv_prep(**dict(prep(), **k))])
def test_scales(call, i):
    with pytest.raises(ValueError, match="scale"):
        call(k_scale=SCALES[i][0], v_scale=SCALES[i][1])


@pytest.mark.parametrize("bad,what", [
    (dict(mask=torch.zeros(B, H, 1, 63)), "mask"),                      # the list holds 64 rows
    (dict(mask=torch.zeros(B + 1, H, 1, 64)), "mask"),
    (dict(mask=torch.zeros(B, 2, 1, 64)), "mask"),
    (dict(mask=torch.zeros(B, H, 2, 64)), "mask"),
    (dict(mask=torch.zeros(B, H, 64)), "mask"),
    (dict(mask=torch.zeros(1, 1, 1, 128)[..., ::2]), "mask"),
    (dict(out=torch.zeros(B, 1, H - 1, D, dtype=torch.float16)), "out"),
    (dict(out=torch.zeros(1, 1, H, D, dtype=torch.float16)), "out"),
    (dict(lse=torch.zeros(B, H - 1, 1)), "lse"),
    (dict(lse=torch.zeros(B, H)), "lse"),
    (dict(head_sink=torch.zeros(H - 1)), "head_sink"),
    (dict(head_sink=torch.zeros(2 * H)[::2]), "head_sink"),
    (dict(k_lens=torch.ones(B + 1, dtype=torch.int32)), "k_lens"),
])
def test_paged_extents(bad, what):
    with pytest.raises(ValueError, match=what):
        attn.decode_paged(**dict(paged(), **bad))


@pytest.mark.parametrize("bad,what", [
    (dict(mask=torch.zeros(B, H, 8, 29)), "mask"),
    (dict(mask=torch.zeros(B, H, 7, 30)), "mask"),
    (dict(mask=torch.zeros(3, 1, 1, 30)), "mask"),
    (dict(lse=torch.zeros(B, H, 7)), "lse"),
    (dict(lse=torch.zeros(B, H, 16)[..., ::2]), "lse"),
    (dict(head_sink=torch.zeros(1)), "head_sink"),
    (dict(k_lens=torch.ones(1, dtype=torch.int32)), "k_lens"),
    (dict(seg=torch.zeros(1, 8, dtype=torch.int32)), "seg"),
    (dict(seg=torch.zeros(B, 7, dtype=torch.int32)), "seg"),
    (dict(seg=torch.zeros(16, dtype=torch.int32)[::2]), "seg"),
    (dict(out=torch.zeros(B, H, 7, D, dtype=torch.float16)), "out"),
    (dict(v=torch.zeros(B, G, 29, D, dtype=torch.float16)), "disagree"),
    (dict(k=torch.zeros(1, G, 30, D, dtype=torch.float16), v=torch.zeros(1, G, 30, D, dtype=torch.float16)), "disagree"),
])
def test_window_extents(bad, what):
    with pytest.raises(ValueError, match=what):
        attn.fwd(**dict(window(), **bad))


@pytest.mark.gpu
def test_types_and_devices():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    i64, cpu = dict(dtype=torch.int64, device="cuda"), dict(dtype=torch.int32)
    good = window("cuda")
    attn.fwd(**good)
    for bad in (dict(k_lens=torch.ones(B, **i64)), dict(k_lens=torch.ones(B, **cpu)), dict(seg=torch.zeros(8, **i64)),
                dict(seg=torch.zeros(B, 8, **cpu)), dict(lse=torch.zeros(B, H, 8, device="cuda").half()),
                dict(lse=torch.zeros(B, H, 8)), dict(head_sink=torch.zeros(H, device="cuda").half()),
                dict(mask=torch.zeros(1, 1, 1, 30)), dict(k=good["k"].cpu())):
        with pytest.raises(ValueError):
            attn.fwd(**dict(good, **bad))
    good = paged("cuda")
    attn.decode_paged(**good, mask=torch.zeros(1, 1, 1, 64, device="cuda"), lse=torch.empty(B, H, 1, device="cuda"))
    attn.decode_paged(**good, mask=torch.zeros(B, H, 1, 50, device="cuda"), max_rows=50)
    for bad in (dict(mask=torch.zeros(1, 1, 1, 64)), dict(mask=torch.zeros(1, 1, 1, 64, device="cuda").half()),
                dict(head_sink=torch.zeros(H)), dict(workspace=torch.empty(1 << 22, dtype=torch.uint8)),
                dict(workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            attn.decode_paged(**dict(good, **bad))
    i8, full = paged("cuda", True), torch.ones(G * D, device="cuda")
    attn.decode_paged(**i8)
    attn.decode_paged(**dict(i8, k_scale=full, v_scale=full))
    with pytest.raises(ValueError):
        attn.decode_paged(**dict(i8, k_scale=full, v_scale=full.double()))
    attn.qkv_prep(**prep("cuda"))
    attn.qkv_prep(**prep("cuda", False))
