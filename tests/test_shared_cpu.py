"""attn_fwd_shared and attn_qkv_prep_axes without a GPU: struct layouts, refusals
(each on the host, before any launch), workspaces and the torch entry points' checks."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from attention_attn_fwd_02_gb300 import attn, build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "attn.h")
FAKE = 0x10000  # never dereferenced: every case below fails on the host first
INVALID, ALIGN, WORKSPACE, UNSUPPORTED = (attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_ALIGNMENT,
                                          attn.ATTN_ERR_WORKSPACE, attn.ATTN_ERR_UNSUPPORTED)


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return attn.lib()


def test_struct_layouts_match_c(tmp_path):
    src, exe = tmp_path / "sz.c", tmp_path / "sz"
    fields = [("attn_prefix", f) for f, _ in attn.attn_prefix._fields_] + \
             [("attn_axes", f) for f, _ in attn.attn_axes._fields_]
    body = "".join(f'printf("%zu\\n", offsetof({t}, {f}));' for t, f in fields)
    src.write_text(f'#include "{HEADER}"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){{'
                   f'printf("%zu\\n%zu\\n", sizeof(attn_prefix), sizeof(attn_axes));{body}return 0;}}\n')
    subprocess.run(["gcc", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = [ctypes.sizeof(attn.attn_prefix), ctypes.sizeof(attn.attn_axes)]
    want += [getattr(getattr(attn, t), f).offset for t, f in fields]
    assert got == want


# ---- attn_fwd_shared -----------------------------------------------------------------------------


def problem(**kw):
    d = dict(batch=2, heads=4, kv_heads=2, q_len=8, k_len=64, head_dim=64, dtype="bf16", causal=True,
             causal_align="klens", q_layout=(0, 2048, 512, 64), k_layout=(0, 2048, 1024, 64),
             v_layout=(0, 2048, 1024, 64), o_layout=(0, 2048, 512, 64))
    d.update(kw)
    return attn.make_problem(d)


PAGES = attn.make_pages(16, 100, FAKE, 4)
PREFIX = attn.make_prefix(500, FAKE)


def call(p, pages=PAGES, prefix=PREFIX, q=FAKE, k=FAKE, v=FAKE, o=FAKE, mask=None, lens=None, lse=None, ws=FAKE,
         n=1 << 40):
    return attn.attn_fwd_shared(p, pages, prefix, q, k, v, o, mask, lens, lse, ws, n, None)


@pytest.mark.parametrize("kw,pages,prefix,code", [
    ({}, PAGES, None, INVALID),
    ({}, None, PREFIX, INVALID),
    ({}, PAGES, attn.make_prefix(-1, FAKE), INVALID),
    ({}, PAGES, attn.make_prefix(1, None), INVALID),
    ({}, PAGES, attn.make_prefix(1, FAKE + 2), ALIGN),
    ({}, PAGES, attn.make_prefix((1 << 30) + 1, FAKE), UNSUPPORTED),
    (dict(k_len=64), PAGES, attn.make_prefix((1 << 30) - 63, FAKE), UNSUPPORTED),   # both together
    (dict(k_len=(1 << 30) + 1), PAGES, PREFIX, UNSUPPORTED),
    (dict(q_len=(1 << 30) + 1), PAGES, PREFIX, UNSUPPORTED),
    ({}, attn.make_pages(0, 100, FAKE, 4), PREFIX, INVALID),
    ({}, attn.make_pages(16, -1, FAKE, 4), PREFIX, INVALID),
    ({}, attn.make_pages(16, 100, None, 4), PREFIX, INVALID),
    ({}, attn.make_pages(16, 100, FAKE + 1, 4), PREFIX, ALIGN),
    ({}, attn.make_pages(16, 100, FAKE, -4), PREFIX, INVALID),
    (dict(window_left=7), PAGES, PREFIX, INVALID),
    (dict(kv_heads=3), PAGES, PREFIX, INVALID),
    (dict(head_dim=63), PAGES, PREFIX, INVALID),
    (dict(head_dim=257), PAGES, PREFIX, INVALID),
    (dict(batch=-1), PAGES, PREFIX, INVALID),
    (dict(softcap=-1.0), PAGES, PREFIX, INVALID),
    (dict(scale=float("inf")), PAGES, PREFIX, INVALID),
    (dict(kv_dtype="i8"), PAGES, PREFIX, INVALID),
    (dict(k_layout=(0, -1, 1, 1)), PAGES, PREFIX, INVALID),
])
def test_refusals(kw, pages, prefix, code):
    p = problem(**kw)
    assert call(p, pages, prefix) == code
    assert attn.attn_fwd_shared_workspace_size(p, pages, prefix) == 0


def test_pointers_and_empty_calls():
    p = problem()
    for name in ("q", "k", "v", "o"):
        assert call(p, **{name: None}) == INVALID, name
        assert call(p, **{name: FAKE + 1}) == ALIGN, name
    for name in ("mask", "lens", "lse"):
        assert call(p, **{name: FAKE + 2}) == ALIGN, name
    own = problem(k_len=0)   # the prefix's keys alone need pools too
    assert call(own, attn.make_pages(16, 100, None, 0), k=None) == INVALID
    assert call(problem(batch=0), q=None, ws=None, n=0) == 0
    assert call(problem(q_len=0), q=None, ws=None, n=0) == 0


@pytest.mark.parametrize("dtype,q_len,head_dim,batch,prefix", [
    ("bf16", 1, 128, 64, 8192), ("f16", 5, 64, 16, 20000), ("bf16", 2048, 128, 3, 4099), ("f32", 1, 128, 60, 6000),
    ("f32", 33, 64, 5, 501), ("bf16", 1, 256, 64, 8192)])
def test_workspace_is_needed(dtype, q_len, head_dim, batch, prefix):
    p = problem(dtype=dtype, q_len=q_len, head_dim=head_dim, batch=batch, heads=32, kv_heads=8, k_len=4096)
    x = attn.make_prefix(prefix, FAKE)
    need = attn.attn_fwd_shared_workspace_size(p, PAGES, x)
    assert need > 0
    assert call(p, prefix=x, ws=None, n=0) == WORKSPACE
    assert call(p, prefix=x, n=need - 1) == WORKSPACE
    assert call(p, prefix=x, ws=FAKE + 16, n=need) == ALIGN


def test_workspace_from_the_shape_alone():
    """Addresses, strides and lengths of a call do not change the size."""
    x = attn.make_prefix(8192, FAKE)
    a = problem(q_len=1, batch=64, heads=32, kv_heads=8, k_len=1024)
    b = problem(q_len=1, batch=64, heads=32, kv_heads=8, k_len=1024, k_layout=(3, 1 << 20, 64, 4096), scale=0.3,
                causal=False)
    other = attn.make_pages(16, 7, FAKE + 64, 900)
    assert attn.attn_fwd_shared_workspace_size(a, PAGES, x) == attn.attn_fwd_shared_workspace_size(b, other, x)


# ---- attn_qkv_prep_axes ---------------------------------------------------------------------------

ARGS = ("q", "k", "v", "q_weight", "k_weight", "cos", "sin", "positions", "rows", "q_out", "k_out", "v_out")


def prep_problem(**kw):
    d = dict(batch=2, seq_len=4, heads=4, kv_heads=2, head_dim=64, rot_dim=64, dtype="bf16", max_pos=16, cache_rows=16,
             q_layout=(0, 1024, 64, 256), k_layout=(0, 512, 64, 128), v_layout=(0, 512, 64, 128),
             q_out_layout=(0, 1024, 64, 256), k_out_layout=(0, 2048, 1024, 64), v_out_layout=(0, 2048, 1024, 64))
    d.update(kw)
    p = attn.make_prep({k: v for k, v in d.items() if k not in ("k_layout_bad",)})
    return p


def call_prep(p, axes, pages=None, **kw):
    a = dict({n: FAKE for n in ARGS}, **kw)
    return attn.lib().attn_qkv_prep_axes(ctypes.byref(p), pages, None if axes is None else ctypes.byref(axes),
                                         *(a[n] for n in ARGS), None)


def test_prep_axes_refusals():
    p, good = prep_problem(), attn.make_axes([0, 1] * 16, 8)
    assert call_prep(p, None) == INVALID
    for axes in (attn.make_axes([0, 4] * 16, 8), attn.make_axes([0, 255] * 16, 8), attn.make_axes([0, 1] * 16, -1),
                 attn.attn_axes(0, 8), attn.attn_axes(5, 8)):
        assert call_prep(p, axes) == INVALID
    low = attn.make_axes([0, 1] * 16, 8)
    low.n_axes = 1   # an axis that is not below n_axes
    assert call_prep(p, low) == INVALID
    for name in ("q", "k", "v", "q_out", "k_out", "v_out", "cos", "sin"):
        assert call_prep(p, good, **{name: None}) == INVALID, name
    for name in ARGS:
        assert call_prep(p, good, **{name: FAKE + 1}) == ALIGN, name
    assert call_prep(prep_problem(rot_dim=63), good) == INVALID
    assert call_prep(prep_problem(max_pos=0), good) == INVALID
    assert call_prep(prep_problem(kv_dtype="i8"), good) == INVALID
    assert call_prep(p, good, attn.make_pages(0, 1, FAKE, 1)) == INVALID
    assert call_prep(prep_problem(batch=0), good, q=None) == 0
    # pairs behind the rotated part have no axis
    tail = attn.make_axes([0, 1] * 8 + [9] * 16, 8)
    tail.n_axes = 2
    assert call_prep(prep_problem(rot_dim=32), tail, q=None) == INVALID and call_prep(prep_problem(rot_dim=32, batch=0),
                                                                                    tail) == 0


def test_make_axes_checks():
    with pytest.raises(ValueError):
        attn.make_axes([0] * 129, 0)
    with pytest.raises(ValueError):
        attn.make_axes([0, -1], 0)


# ---- the torch entry points: extents, with host tensors -----------------------------------------------


def test_fwd_shared_extents():
    torch = pytest.importorskip("torch")
    B, H, G, D, ps = 2, 4, 2, 64, 16
    f16 = dict(dtype=torch.float16)
    good = dict(q=torch.zeros(B, 3, H, D, **f16), k_pool=torch.zeros(8, G, ps, D, **f16),
                v_pool=torch.zeros(8, G, ps, D, **f16), prefix_table=torch.zeros(3, dtype=torch.int32), prefix_rows=40,
                table=torch.zeros(B, 4, dtype=torch.int32))
    for bad, what in ((dict(prefix_rows=49), "prefix_table"), (dict(prefix_rows=-1), "prefix_table"),
                      (dict(prefix_table=torch.zeros(1, 3, dtype=torch.int32)), "prefix_table"),
                      (dict(prefix_table=torch.zeros(6, dtype=torch.int32)[::2]), "prefix_table"),
                      (dict(max_rows=65), "max_rows"), (dict(q=torch.zeros(B, H, D, **f16)), "q"),
                      (dict(table=torch.zeros(B + 1, 4, dtype=torch.int32)), "disagree"),
                      (dict(v_pool=torch.zeros(7, G, ps, D, **f16)), "disagree"),
                      (dict(mask=torch.zeros(B, H, 3, 103)), "mask"), (dict(mask=torch.zeros(B, H, 2, 104)), "mask"),
                      (dict(lse=torch.zeros(B, H, 2)), "lse"), (dict(head_sink=torch.zeros(H - 1)), "head_sink"),
                      (dict(k_lens=torch.ones(B + 1, dtype=torch.int32)), "k_lens"),
                      (dict(out=torch.zeros(B, 3, H - 1, D, **f16)), "out"),
                      (dict(k_pool=torch.zeros(8, G, ps, D, dtype=torch.int8),
                            v_pool=torch.zeros(8, G, ps, D, dtype=torch.int8)), "scale"), ({}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            attn.fwd_shared(**dict(good, **bad))
