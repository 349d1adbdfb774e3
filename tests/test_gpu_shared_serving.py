"""A layer as a server of many questions about one image or video runs it:
positions on three axes prepare the image's tokens into pages that every question
then shares, the questions' own prompts and the tokens after them."""
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


def serve(dt, grid, questions, steps, *, H=8, G=2, D=128, ps=16, graph=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    half = D // 2
    axes = [0] * (half // 4) + [1] * (3 * half // 8) + [2] * (half - half // 4 - 3 * half // 8)
    n_img = grid[0] * grid[1] * grid[2]
    B, S = len(questions), max(questions)
    room = S + steps
    width, img_pages = -(-room // ps), -(-n_img // ps)
    perm = torch.randperm(B * width + img_pages, generator=g, device="cuda").to(torch.int32)
    table, prefix = perm[:B * width].view(B, width).contiguous(), perm[B * width:].contiguous()
    kc, vc = (torch.full((perm.numel(), G, ps, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    ang = torch.arange(max(grid) + room, device="cuda")[:, None] * 100.0 ** -torch.linspace(0, 1, half, device="cuda")
    norms = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2)]
    common = dict(q_weight=norms[0], k_weight=norms[1], cos=ang.cos(), sin=ang.sin(), axes=axes)
    draw = lambda *s: torch.randn(*s, H + 2 * G, D, generator=g, device="cuda").to(dt)  # noqa: E731
    split = lambda t: (t[:, :, :H], t[:, :, H:H + G], t[:, :, H + G:])  # noqa: E731
    # the image: one entry, its pages the prefix's
    at = torch.arange(n_img, device="cuda")
    pos = torch.stack([at // (grid[1] * grid[2]), at // grid[2] % grid[1], at % grid[2]])[:, None].to(torch.int32)
    rows = at[None].to(torch.int32)
    attn.qkv_prep(*split(draw(1, n_img)), kc, vc, prefix[None].contiguous(), positions=pos.contiguous(), rows=rows,
                  **common)
    # the questions: text has one position on every axis; padding tokens in front write nothing
    n = torch.tensor(questions, device="cuda")
    i = torch.arange(S, device="cuda")[None] - (S - n)[:, None]
    tpos = torch.where(i >= 0, max(grid) + i, 0).to(torch.int32).expand(3, B, S).contiguous()
    q = attn.qkv_prep(*split(draw(B, S)), kc, vc, table, positions=tpos, rows=torch.where(i >= 0, i, -1).to(torch.int32),
                      **common)
    lens = n.to(torch.int32)
    args = (kc, vc, prefix, n_img, table)
    out = attn.fwd_shared(q, *args, lens, max_rows=room)
    seen = [(q, lens.clone(), out)]
    xs = [draw(B, 1) for _ in range(steps)]
    xin, qbuf, obuf = torch.empty_like(xs[0]), torch.empty_like(q[:, :1].contiguous()), torch.empty_like(q[:, :1].contiguous())
    ppos, prow = torch.empty(3, B, 1, dtype=torch.int32, device="cuda"), torch.empty(B, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def step():
        prow.copy_(lens[:, None])
        ppos.copy_((max(grid) + prow).expand(3, B, 1))
        attn.qkv_prep(*split(xin), kc, vc, table, positions=ppos, rows=prow, out=qbuf, **common)
        lens.add_(1)
        attn.fwd_shared(qbuf, *args, lens, max_rows=room, workspace=ws, out=obuf)

    run = step
    if graph:
        keep = [t.clone() for t in (lens, kc, vc)]
        xin.copy_(xs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for t, k in zip((lens, kc, vc), keep):
            t.copy_(k)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        run = cg.replay
    for x in xs:
        xin.copy_(x)
        run()
        seen.append((qbuf.clone(), lens.clone(), obuf.clone()))
    return dict(seen=seen, kc=kc, vc=vc, prefix=prefix, n_img=n_img, table=table, ps=ps, room=room, S=S)


@pytest.mark.parametrize("dt,grid,questions", [
    ("bf16", (3, 11, 13), [40, 7, 1, 33]), ("f16", (4, 20, 24), [3, 60]), ("f32", (2, 9, 8), [20, 5, 11]),
    ("bf16", (8, 40, 40), [(3 * b) % 17 + 1 for b in range(30)])])
def test_questions_about_one_image(dt, grid, questions):
    r = serve(DT[dt], grid, questions, 4)
    P = r["n_img"]
    pk, pv = (sb.rows_of(r[x], r["prefix"][None], r["ps"], P) for x in ("kc", "vc"))
    ok, ov = (sb.rows_of(r[x], r["table"], r["ps"], r["room"]) for x in ("kc", "vc"))
    for s, (q, lens, out) in enumerate(r["seen"]):
        Sq = q.shape[1]
        diag = torch.arange(Sq, device="cuda") + (lens[:, None] - Sq)
        vis = torch.arange(r["room"], device="cuda") <= diag[..., None]
        for b in range(0, len(questions), max(1, len(questions) // 4)):
            k, v = (torch.cat([x, y[b:b + 1]], 2) for x, y in ((pk, ok), (pv, ov)))
            see = torch.cat([torch.ones(1, Sq, P, dtype=torch.bool, device="cuda"), vis[b:b + 1]], 2)
            o, _, tol, _ = sb.attention(q[b:b + 1].transpose(1, 2), k, v, see, p="single")
            sb.check(out[b:b + 1].transpose(1, 2), o, tol, f"step {s}, entry {b}")
    assert attn.attn_device_status(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK


@pytest.mark.parametrize("questions", [[40, 7, 1], [(3 * b) % 17 + 1 for b in range(60)]])
def test_captured_steps_give_the_same_bits(questions):
    a, b = (serve(torch.bfloat16, (4, 30, 30), questions, 4, graph=x) for x in (False, True))
    for x, y in zip(a["seen"], b["seen"]):
        assert all(torch.equal(s, t) for s, t in zip(x, y))
    assert torch.equal(torch.nan_to_num(a["kc"]), torch.nan_to_num(b["kc"]))
