"""Calls of the torch entry points on a stream given as `stream=`: what a call
allocates is that stream's, so no later allocation of another stream gets the
memory while the kernels run, and calls side by side leave one another alone."""
from __future__ import annotations

import pytest

from attention_attn_fwd_02_gb300 import attn, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    attn.lib()


def half(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").half()


def paged_job(seed, B=58, H=8, G=8, rows=1800):
    """Lists that are cut into shares: fragments and notes of cuts in the workspace."""
    q, k, v = half(B, 1, H, 64, seed=seed), half(60, G, 16, 64, seed=seed + 1), half(60, G, 16, 64, seed=seed + 2)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = torch.randint(0, 60, (B, rows // 16), generator=g, device="cuda").to(torch.int32)
    n = torch.randint(rows // 3, rows, (B,), generator=g, device="cuda").to(torch.int32)
    return lambda **kw: attn.decode_paged(q, k, v, table, n, **kw)


def window_job(seed):
    q, kv = half(1, 2, 100, 64, seed=seed), half(1, 2, 4000, 64, seed=seed + 1)
    return lambda **kw: attn.fwd(q, kv, kv, layout="bhsd", causal=True, window_left=3000, first_keys=4, key_splits=7, **kw)


def fwd_job(seed):
    q, kv = half(1, 2, 100, 64, seed=seed), half(1, 2, 9000, 64, seed=seed + 1)
    return lambda **kw: attn.fwd(q, kv, kv, layout="bhsd", **kw)


def decode_job(seed):
    q, kv = half(4, 1, 8, 128, seed=seed), half(4, 2, 5000, 128, seed=seed + 1)
    return lambda **kw: attn.decode(q, kv, kv, **kw)


def combine_job(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    o, lse = torch.randn(500, 4, 64, generator=g, device="cuda"), torch.randn(500, 4, generator=g, device="cuda")
    return lambda **kw: attn.combine(o, lse, **kw)


JOBS = dict(paged=(paged_job, "attn_decode_paged"), window=(window_job, "attn_fwd_window"), fwd=(fwd_job, "attn_fwd"),
            decode=(decode_job, "attn_decode"))


@pytest.mark.parametrize("name", JOBS)
def test_workspace_belongs_to_the_stream(name, monkeypatch):
    """Nothing is launched here: the entry point is replaced by a note of its workspace."""
    make, entry = JOBS[name]
    job, st, seen = make(3), torch.cuda.Stream(), []
    monkeypatch.setattr(attn, entry, lambda *a: seen.append((a[-3], a[-2])) or 0)
    torch.cuda.synchronize()
    out = job(stream=st.cuda_stream)
    ws, size = seen[0]
    assert ws and size
    torch.cuda.synchronize()
    later = torch.empty(size, dtype=torch.uint8, device="cuda")
    lo, hi = later.data_ptr(), later.data_ptr() + size
    assert not (lo < ws + size and ws < hi), "the current stream was given the workspace of a call on another stream"
    with torch.cuda.stream(st):   # that stream has it
        assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() == ws
    del out


@pytest.mark.parametrize("name", [*JOBS, "combine"])
def test_calls_side_by_side(name):
    jobs = [JOBS[name][0](s) if name in JOBS else combine_job(s) for s in (10, 20, 30)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], []
    for _ in range(8):
        for st, j in zip(streams, jobs):
            got.append(j(stream=st.cuda_stream))
            torch.empty(1 << 21, dtype=torch.uint8, device="cuda").fill_(255)   # the current stream's own work
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 3])


@pytest.mark.parametrize("name", [*JOBS, "combine"])
def test_names_of_the_default_stream(name):
    job = JOBS[name][0](5) if name in JOBS else combine_job(5)
    want = job()
    for st in (0, 1):
        assert torch.equal(job(stream=st), want)


def test_given_stream_under_capture():
    job = paged_job(40)
    want = job()
    st = torch.cuda.Stream()
    job(stream=st.cuda_stream)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = job(stream=st.cuda_stream)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
