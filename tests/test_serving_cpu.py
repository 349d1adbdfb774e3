"""attn_fwd_window, attn_decode_paged and attn_qkv_prep without a GPU: struct
layouts, refusals (each on the host, before any launch) and workspace plans."""
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
    fields = [("attn_pages", f) for f, _ in attn.attn_pages._fields_] + \
             [("attn_prep", f) for f, _ in attn.attn_prep._fields_]
    body = "".join(f'printf("%zu\\n", offsetof({t}, {f}));' for t, f in fields)
    src.write_text(f'#include "{HEADER}"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){{'
                   f'printf("%zu\\n%zu\\n", sizeof(attn_pages), sizeof(attn_prep));{body}return 0;}}\n')
    subprocess.run(["gcc", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = [ctypes.sizeof(attn.attn_pages), ctypes.sizeof(attn.attn_prep)]
    want += [getattr(getattr(attn, t), f).offset for t, f in fields]
    assert got == want


# ---- attn_fwd_window -----------------------------------------------------------------------------


def window_problem(**kw):
    d = dict(batch=2, heads=4, kv_heads=2, q_len=8, k_len=64, head_dim=64, dtype="bf16", causal=True, window_left=15,
             q_layout=(0, 2048, 512, 64), k_layout=(0, 8192, 4096, 64), v_layout=(0, 8192, 4096, 64),
             o_layout=(0, 2048, 512, 64))
    d.update(kw)
    return attn.make_problem(d)


def call_window(p, first, q=FAKE, k=FAKE, v=FAKE, o=FAKE, mask=None, ws=None, n=0):
    return attn.attn_fwd_window(p, first, q, k, v, o, mask, None, None, None, ws, n, None)


@pytest.mark.parametrize("kw,first,code", [
    ({}, -1, INVALID),
    ({}, (1 << 30) + 1, INVALID),
    (dict(window_left=-1), 4, INVALID),
    (dict(window_left=-1, causal=False), 4, INVALID),
    (dict(window_left=-1), 0, INVALID),              # a window operator without a window
    (dict(kv_heads=3), 4, INVALID),
    (dict(head_dim=63), 4, INVALID),
    (dict(k_len=(1 << 30) + 1), 4, UNSUPPORTED),
])
def test_window_refusals(kw, first, code):
    assert call_window(window_problem(**kw), first) == code
    assert attn.attn_fwd_window_workspace_size(window_problem(**kw), first) == 0


def test_window_pointers_and_empty_calls():
    p = window_problem()
    for name in "qkvo":
        assert call_window(p, 4, **{name: None}) == INVALID
        assert call_window(p, 4, **{name: FAKE + 1}) == ALIGN
    assert call_window(p, 4, mask=FAKE + 2) == ALIGN
    assert call_window(window_problem(batch=0), 4, None, None, None, None) == 0
    assert call_window(window_problem(q_len=0), 4, None, None, None, None) == 0


def _r256(x):
    return (x + 255) // 256 * 256


def _parts(B, H, G, Sq, Sk, D, w, first, ks):
    """The float32 plan's cost model, restated: waves of one CTA an SM with their part of the tiles, and the merge.
    (The half types' own parts are clusters, which take no workspace.)"""
    if ks:
        return min(ks, 16)
    blocks = -(-Sq * H // G // 32) * G * B
    if blocks >= 304:
        return 1
    tiles = -(-min(Sk, w + first + 32) // 32) + 1

    def cost(n):
        return -(-blocks * n // 152) * -(-tiles // n) * 2.1 * D / 128 + (n > 1) * (4.0 + blocks * 32 * n * D * 8 / 6.5e6)

    return min(range(1, min(16, tiles) + 1), key=cost)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Sq,Sk,D,w,first,ks", [
    (1, 4, 64, 20000, 128, 4095, 64, 0), (1, 4, 64, 20000, 128, 255, 4, 0), (2, 32, 4096, 4096, 128, 1023, 4, 0),
    (1, 2, 100, 5000, 256, 5000, 10, 0), (1, 2, 100, 500, 64, 63, 2, 5), (1, 1, 9, 900, 64, 63, 2, 40)])
def test_window_workspace_follows_the_plan(B, H, Sq, Sk, D, w, first, ks, dtype):
    p = window_problem(dtype=dtype, batch=B, heads=H, kv_heads=1, q_len=Sq, k_len=Sk, head_dim=D, window_left=w, key_splits=ks)
    n = _parts(B, H, 1, Sq, Sk, D, w, first, ks) if dtype == "f32" or ks else 1
    rows = B * H * Sq
    assert attn.attn_fwd_window_workspace_size(p, first) == (0 if n == 1 else _r256(rows * n * D * 4) +
                                                             _r256(rows * n * 4))


def test_window_forced_parts_need_the_workspace():
    p = window_problem(key_splits=3)
    need = attn.attn_fwd_window_workspace_size(p, 4)
    assert call_window(p, 4) == WORKSPACE
    assert call_window(p, 4, ws=FAKE, n=need - 1) == WORKSPACE
    assert call_window(p, 4, ws=FAKE + 16, n=need) == ALIGN


# ---- attn_decode_paged ---------------------------------------------------------------------------


def paged_problem(**kw):
    d = dict(batch=2, heads=4, kv_heads=2, q_len=1, k_len=4096, head_dim=64, dtype="bf16",
             q_layout=(0, 256, 64, 64), k_layout=(0, 2048, 1024, 64), v_layout=(0, 2048, 1024, 64),
             o_layout=(0, 256, 64, 64))
    d.update(kw)
    return attn.make_problem(d)


def call_paged(p, pages, first=0, q=FAKE, k=FAKE, v=FAKE, o=FAKE, ws=FAKE, n=1 << 40):
    return attn.attn_decode_paged(p, pages, first, q, k, v, o, None, None, None, ws, n, None)


PAGES = dict(page_size=16, n_pages=10, table=FAKE, table_stride=256)


@pytest.mark.parametrize("kw,pg,first,code", [
    (dict(q_len=2), {}, 0, INVALID),
    ({}, dict(page_size=0), 0, INVALID),
    ({}, dict(page_size=-4), 0, INVALID),
    ({}, dict(n_pages=-1), 0, INVALID),
    ({}, dict(table_stride=-1), 0, INVALID),
    ({}, dict(table=None), 0, INVALID),
    ({}, dict(table=FAKE + 2), 0, ALIGN),
    ({}, {}, -1, INVALID),
    ({}, {}, 4, INVALID),                               # first keys without a window
    (dict(kv_dtype="i8"), {}, 0, INVALID),              # int8 pools need their scales
    (dict(heads=5), {}, 0, INVALID),
    (dict(k_len=(1 << 30) + 1), {}, 0, UNSUPPORTED),
])
def test_paged_refusals(kw, pg, first, code):
    p, pages = paged_problem(**kw), attn.make_pages(**dict(PAGES, **pg))
    assert call_paged(p, pages, first) == code
    assert attn.attn_decode_paged_workspace_size(p, pages, first) == 0


def test_paged_pointers_workspace_and_empty_calls():
    p, pages = paged_problem(), attn.make_pages(**PAGES)
    assert call_paged(p, None) == INVALID
    for name in "qkvo":
        assert call_paged(p, pages, **{name: None}) == INVALID
        assert call_paged(p, pages, **{name: FAKE + 1}) == ALIGN
    need = attn.attn_decode_paged_workspace_size(p, pages, 0)
    assert need > 0 and need % 256 == 0
    assert call_paged(p, pages, ws=None) == WORKSPACE
    assert call_paged(p, pages, n=need - 1) == WORKSPACE
    assert call_paged(p, pages, ws=FAKE + 16, n=need) == ALIGN
    assert call_paged(paged_problem(batch=0), pages, q=None, o=None, ws=None, n=0) == 0


# ---- attn_qkv_prep -------------------------------------------------------------------------------


def prep_problem(**kw):
    d = dict(batch=2, seq_len=3, heads=4, kv_heads=2, head_dim=64, rot_dim=64, dtype="bf16", max_pos=100,
             cache_rows=100, q_layout=(0, 1536, 64, 512), k_layout=(256, 1536, 64, 512),
             v_layout=(384, 1536, 64, 512), q_out_layout=(0, 768, 64, 256), k_out_layout=(0, 12800, 6400, 64),
             v_out_layout=(0, 12800, 6400, 64))
    d.update(kw)
    return attn.make_prep(d)


ARGS = dict(q=FAKE, k=FAKE, v=FAKE, q_weight=None, k_weight=None, cos=FAKE, sin=FAKE, positions=None, rows=None,
            q_out=FAKE, k_out=FAKE, v_out=FAKE)


def call_prep(p, pages=None, **kw):
    return attn.attn_qkv_prep(p, pages, *dict(ARGS, **kw).values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(seq_len=-1), INVALID), (dict(heads=3), INVALID), (dict(kv_heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=258), INVALID), (dict(head_dim=63, rot_dim=2), INVALID),
    (dict(rot_dim=3), INVALID), (dict(rot_dim=66), INVALID), (dict(rot_dim=-2), INVALID), (dict(dtype=3), INVALID),
    (dict(interleaved=2), INVALID), (dict(norm=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(max_pos=0), INVALID),
    (dict(cache_rows=-1), INVALID), (dict(k_layout=(0, -1, 1, 1)), INVALID), (dict(row_batch_stride=-1), INVALID),
    (dict(kv_dtype="i8"), INVALID), (dict(kv_dtype="i8", k_scale_ptr=FAKE, v_scale_ptr=FAKE + 1), ALIGN),
])
def test_prep_refusals(kw, code):
    assert call_prep(prep_problem(**kw)) == code


def test_prep_pointers_and_empty_calls():
    p = prep_problem()
    for name in ("q", "k", "v", "q_out", "k_out", "v_out", "cos", "sin"):
        assert call_prep(p, **{name: None}) == INVALID, name
    for name in ARGS:
        assert call_prep(p, **{name: FAKE + 1}) == ALIGN, name
    assert call_prep(p, attn.make_pages(0, 1, FAKE, 1)) == INVALID
    assert call_prep(p, attn.make_pages(16, 1, None, 1)) == INVALID
    assert call_prep(prep_problem(batch=0), q=None) == 0
    assert call_prep(prep_problem(seq_len=0), q=None) == 0
