"""What attn_fwd_shared_workspace_size depends on: the fields that the header names and no others."""
from __future__ import annotations

import os
import random
import re

import pytest

from attention_attn_fwd_02_gb300 import attn, build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "attn.h")
FAKE = 0x10000  # never dereferenced

# Other values of each field than those of `shapes` below.
OTHERS = dict(
    scale=[0.3, -1.0, 3e38], causal=[False], masked_rows=["zero"],
    k_layout=[(3, 1 << 20, 64, 4096)], q_layout=[(5, 1 << 20, 64, 4096)], mask_layout=[(0, 9, 8, 7)], lse_layout=[(3, 2)],
    k_lens_kind=["last_index"], softcap=[2.0], smooth_softmax=[True], head_sink_ptr=[FAKE], key_splits=[3],
    page_size=[8, 64, 7], n_pages=[1, 900], table=[FAKE + 64], table_stride=[900], prefix_table=[FAKE + 128])
FIXED = dict(causal_align="fixed", causal_offset=-100)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    attn.lib()


def size(**kw):
    d = dict(q_layout=(0, 1 << 24, 512, 64), k_layout=(0, 1 << 24, 1024, 64), v_layout=(0, 1 << 24, 1024, 64),
             o_layout=(0, 1 << 24, 512, 64), causal=True, causal_align="klens", page_size=16, n_pages=100, table=FAKE,
             table_stride=4, prefix_table=FAKE)
    d.update(kw)
    pages = attn.make_pages(d["page_size"], d["n_pages"], d["table"], d["table_stride"])
    prefix = attn.make_prefix(d["prefix"], d["prefix_table"])
    p = attn.make_problem(d)
    got = attn.attn_fwd_shared_workspace_size(p, pages, prefix)
    if got:   # a byte less is refused on the host
        assert attn.attn_fwd_shared(p, pages, prefix, FAKE, FAKE, FAKE, FAKE, None, None, None, FAKE, got - 1,
                                    None) == attn.ATTN_ERR_WORKSPACE
    return got


def shapes(n):
    r = random.Random(7)
    for i in range(n):
        g = r.choice([1, 2, 4, 8])
        yield dict(batch=r.randint(1, 40), heads=g * r.choice([1, 2, 3, 4]), kv_heads=g,
                   q_len=r.choice([1, r.randint(2, 12), r.randint(13, 700)]), k_len=r.randint(0, 2000),
                   head_dim=r.choice([64, 128, 128, 80, 256]), dtype=r.choice(["bf16", "f16", "f32"]),
                   prefix=r.choice([0, r.randint(1, 500), r.randint(501, 20000)]))


def test_the_header_names_what_changes_the_size():
    text = open(HEADER).read()
    said = re.search(r"/\* Bytes of device workspace attn_fwd_shared needs.*?\*/", text, re.S).group(0)
    changed = {False: set(), True: set()}   # by q_len > 1
    for kw in shapes(250):
        at = size(**kw)
        for name, values in OTHERS.items():
            if any(size(**dict(kw, **{name: v})) != at for v in values):
                changed[kw["q_len"] > 1].add(name)
        fixed = size(**kw, **FIXED)
        for name, moved in (("causal_align", fixed != at),
                            ("causal_offset", fixed != size(**dict(kw, **FIXED) | dict(causal_offset=300)))):
            if moved:
                changed[kw["q_len"] > 1].add(name)
    assert changed[False] <= {"page_size"}
    causal = {"causal", "causal_align", "causal_offset"}
    assert causal <= changed[True] <= causal | {"page_size"}
    for name in changed[False] | changed[True]:
        assert re.search(rf"\b{name}\b", said), name


def test_a_size_of_one_causal_setting_may_not_do_for_another():
    kw = dict(batch=1, heads=4, kv_heads=1, q_len=200, k_len=1200, head_dim=128, dtype="bf16", prefix=1000)
    sizes = [size(**kw, **c) for c in ({}, dict(causal=False), dict(causal_align="fixed", causal_offset=0))]
    assert len(set(sizes)) == 3
