"""GPU parity of lora_fused_gemm_w4 and lora_fused_glu / _fp8w / _w4 against the
fp64 definitions: every weight type and group, token counts around the 16-token
blocks, the 64-token chunks and the 256-token tiles, odd widths, padded rows,
every kind of id, and the calls a serving loop makes (graphs, streams)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import segmented_gathered_rank_amd as sgr  # noqa: E402
from base_util import SENTINEL, Problem  # noqa: E402

FORMS = [("gemm", "int4", 32), ("gemm", "int4", 64), ("gemm", "int4", 128), ("gemm", "int4z", 32),
         ("gemm", "int4z", 64), ("gemm", "int4z", 128), ("gemm", "table", 32), ("gemm", "table", 64),
         ("gemm", "table", 128), ("glu", "bf16", 0), ("glu", "fp8", 0), ("glu", "int4", 64), ("glu", "int4z", 32),
         ("glu", "int4z", 128), ("glu", "table", 32), ("glu", "table", 64), ("glu", "table", 128)]
IDS = [f"{o}-{k}-{g}" for o, k, g in FORMS]


def _run(*a, **kw):
    p = Problem(*a, **kw)
    p.call()
    p.check(what=str(a))
    p.close()


@pytest.mark.parametrize("op,kind,group", FORMS, ids=IDS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 64, 65, 130, 300])
def test_token_counts(op, kind, group, n):
    """Ranks 1..64 in one batch, one empty slot, ids of every slot and -1."""
    _run(op, kind, n, 384, 320, group=group or 64, ranks=(16, 3, 64, 0, 17), act="silu", seed=n)


@pytest.mark.parametrize("op,kind,group", FORMS, ids=IDS)
@pytest.mark.parametrize("n", [5, 70, 260])
@pytest.mark.parametrize("h_in,h_out", [(128, 64), (640, 192), (1152, 448)])
def test_widths_and_padded_rows(op, kind, group, n, h_in, h_out):
    """Widths that end inside a tile, a step and a load; rows padded by NaN (x, bf16 weights, fp8
    codes) and by other codes; zero points up to 255."""
    _run(op, kind, n, h_in, h_out, group=group or 64, ranks=(8, 24), act="gelu", pads=3, seed=h_in + n)


@pytest.mark.parametrize("op,kind,group", [f for f in FORMS if f[2] != 128], ids=[i for i in IDS if "128" not in i])
@pytest.mark.parametrize("n", [3, 40, 200])
def test_half_load_tail(op, kind, group, n):
    """h_in an odd multiple of 64: a row of 4-bit codes ends inside a 128-k load."""
    _run(op, kind, n, 64 * 7, 128, group=group or 64, ranks=(16,), act="gelu_tanh", seed=n)
    _run(op, kind, n, 64, 64, group=group or 64, ranks=(64,), act="gelu_tanh", seed=n + 1)


@pytest.mark.parametrize("op,kind,group", [("gemm", "int4z", 64), ("gemm", "table", 128), ("glu", "bf16", 0),
                                           ("glu", "fp8", 0), ("glu", "int4", 32)])
@pytest.mark.parametrize("n", [9, 64, 129, 290])
@pytest.mark.parametrize("ids", ["none", "bad", "runs", "one", "null"])
def test_kinds_of_ids(op, kind, group, n, ids):
    """No token with an adapter, ids out of range on both sides, runs, one adapter for all, no ids."""
    _run(op, kind, n, 256, 192, group=group or 64, ranks=(16, 33, 5), ids=ids, seed=n)


@pytest.mark.parametrize("n", [11, 280])
def test_every_token_its_own_adapter(n):
    _run("gemm", "int4", n, 256, 128, ranks=(4,) * n, ids=np.arange(n)[::-1].copy(), seed=1)
    _run("glu", "bf16", n, 256, 128, ranks=(4,) * n, ids=np.arange(n)[::-1].copy(), seed=2)


@pytest.mark.parametrize("n", [6, 300])
@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_adapter_on_one_projection_only(n, kind):
    """Slots loaded for the gate alone, the up projection alone, both and neither."""
    _run("glu", kind, n, 256, 192, ranks=(16, 16, 16, 16), load=lambda s, p: (s >> p) & 1 == 1, seed=7)


@pytest.mark.parametrize("n", [6, 300])
def test_one_module_for_both_projections(n):
    p = Problem("glu", "bf16", n, 256, 192, ranks=(16, 7), seed=8)
    p.call(modules=(1, 1))
    p.check(modules=(1, 1))
    p.call(modules=(1, 0))
    p.check(modules=(1, 0))
    p.close()


@pytest.mark.parametrize("page,h_in,h_out", [(320, 960, 640), (64, 1984, 128), (192, 192, 1536), (832, 4160, 832)])
@pytest.mark.parametrize("n", [4, 90])
def test_pages(page, h_in, h_out, n):
    """Rank rows over many pages (up to 31) and one, pages that no tile width divides."""
    _run("gemm", "int4", n, h_in, h_out, page=page, group=64, ranks=(64, 5), seed=page)
    _run("glu", "fp8", n, h_in, h_out, page=page, ranks=(20, 5), seed=page + 1)


@pytest.mark.parametrize("op,kind", [("gemm", "int4z"), ("gemm", "table"), ("glu", "bf16"), ("glu", "fp8"), ("glu", "table")])
@pytest.mark.parametrize("n", [20, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_rows_stay_in_their_rows(op, kind, n, bad):
    """A row of x with an infinity or NaN gives non-finite outputs; every other row is as without it."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(n, 256))
    clean = Problem(op, kind, n, 256, 192, group=32, ranks=(16, 8), seed=4, x=x)
    clean.call()
    torch.cuda.synchronize()
    x2 = x.copy()
    x2[n // 2, 100] = bad
    p = Problem(op, kind, n, 256, 192, group=32, ranks=(16, 8), seed=4, x=x2)
    p.call()
    torch.cuda.synchronize()
    keep = np.arange(n) != n // 2
    assert torch.equal(p.y[:n][keep].view(torch.int16), clean.y[:n][keep].view(torch.int16))
    assert not torch.isfinite(p.y[n // 2, :192]).all()
    if op == "gemm":
        assert not torch.isfinite(p.y[n // 2, :192]).any()
    clean.close()
    p.close()


def _rows_of(p, tokens):
    """The problem's reference at some tokens only."""
    x, ids = p.x64, p.ids64
    p.x64, p.ids64 = x[tokens], ids[tokens]
    v, bound = p.reference()
    p.x64, p.ids64 = x, ids
    return v, bound


@pytest.mark.parametrize("op,kind,h_in,h_out,n", [("gemm", "int4", 1024, 1024, 64 * 256 + 40),
                                                   ("gemm", "table", 1024, 1024, 64 * 256),
                                                   ("glu", "fp8", 2048, 1024, 16 * 256 + 200),
                                                   ("glu", "bf16", 512, 2048, 8 * 256 + 1)])
def test_long_batches_and_their_rest(op, kind, h_in, h_out, n):
    """Several rounds of tiles, and a rest past a multiple of 256 that goes another way; sampled
    tokens around every seam, and nothing written behind the last."""
    p = Problem(op, kind, n, h_in, h_out, page=256, group=128, ranks=(16, 33, 0, 7), ids="runs", seed=21, w_scale=0.02)
    p.call()
    torch.cuda.synchronize()
    got = p.y.double().cpu().numpy()
    assert np.all(got[n:] == SENTINEL)
    rng = np.random.default_rng(1)
    toks = np.unique(np.concatenate([np.arange(min(n, 300)), np.arange(n // 256 * 256 - 20, n),
                                     rng.integers(0, n, 200)]))
    v, bound = _rows_of(p, toks)
    assert np.all(np.abs(got[toks] - v) <= bound)
    p.close()


@pytest.mark.parametrize("n", [40, 1000, 2100])
@pytest.mark.parametrize("share", [0.0, 0.5])
def test_smaller_workspaces(n, share):
    """Without ids any workspace will do, none among them; with ids a shorter one than asked for
    either limits the split of h_in or is refused, and never changes what is computed."""
    p = Problem("gemm", "int4z", n, 2048, 256, page=256, group=64, ranks=(16, 5), seed=22)
    nb = sgr.lora_fused_workspace_bytes(p.pool, 0, 1, n)
    ws = torch.full((max(int(nb * share) // 16 * 4, 4),), float("nan"), device="cuda")
    try:
        p.call(ws=ws)
        p.check()
    except sgr.LoraError as e:
        assert e.status == -9
        torch.cuda.synchronize()
        assert bool((p.y == SENTINEL).all())
    ids, p.ids, p.ids64 = p.ids, None, None
    sgr.lora_fused_gemm_w4(p.pool, 0, p.x, p.ld_x, p.wdev[0], None, n, p.y, p.ld_y, ws if share else None)
    p.check()
    p.close()


def _least_workspace(p):
    """Base sums of one split and t, fp32: with it h_in is not split over workgroups."""
    return torch.full((p.np * p.n * (p.h_out + 64),), float("nan"), device="cuda")


@pytest.mark.parametrize("op,kind,group", FORMS, ids=IDS)
@pytest.mark.parametrize("n", [1, 9, 16])
@pytest.mark.parametrize("ws", ["least", "asked for", "none"])
def test_wide_rows_of_few_tokens(op, kind, group, n, ws):
    """h_in past what LDS holds of x (the 64-token kernel with one block of 16), and the same split
    into ranges that LDS does hold; h_in ends half way into the last 128 where the group allows."""
    h_in, page = (4224, 384) if group == 128 else (4160, 320)
    p = Problem(op, kind, n, h_in, 4 * page, group=group or 64, page=page, ranks=(16, 40, 0, 9), seed=31 + n,
                ids="null" if ws == "none" else "random", w_scale=0.02)
    if ws == "none":
        p.ws = torch.empty(0, device="cuda")
    p.call(ws=_least_workspace(p) if ws == "least" else None)
    p.check(what=ws)
    p.close()


@pytest.mark.parametrize("op,kind,group", FORMS, ids=IDS)
@pytest.mark.parametrize("n", [24, 48, 60])
@pytest.mark.parametrize("ws", ["least", "asked for"])
def test_wide_rows_of_more_tokens(op, kind, group, n, ws):
    """Every count of 16-token blocks over more steps of h_in than are held at a time, whole and split."""
    h_in, page = (2176, 128) if group == 128 else (2240, 320)
    p = Problem(op, kind, n, h_in, 5 * page, group=group or 64, page=page, ranks=(16, 64, 0, 9), seed=41 + n, w_scale=0.02)
    p.call(ws=_least_workspace(p) if ws == "least" else None)
    p.check(what=ws)
    p.close()


@pytest.mark.parametrize("op,kind", [("gemm", "int4"), ("glu", "bf16"), ("glu", "fp8"), ("glu", "table")])
def test_zero_tokens(op, kind):
    p = Problem(op, kind, 4, 128, 64, ranks=(8,))
    p.call(n=0)
    torch.cuda.synchronize()
    assert bool((p.y == SENTINEL).all())
    p.close()


@pytest.mark.parametrize("op,kind,n", [("gemm", "int4", 5), ("gemm", "table", 300), ("glu", "bf16", 3), ("glu", "int4z", 64),
                                       ("glu", "fp8", 270)])
def test_same_bits_every_time_and_on_another_stream(op, kind, n):
    p = Problem(op, kind, n, 512, 320, ranks=(16, 40, 9), seed=9)
    p.call()
    torch.cuda.synchronize()
    first = p.y.clone()
    other = torch.cuda.Stream()
    for stream in (None, other, other):
        p.y.fill_(SENTINEL)
        torch.cuda.synchronize()
        p.call(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(p.y, first)
    p.check()
    p.close()


@pytest.mark.parametrize("op,kind", [("gemm", "int4"), ("glu", "fp8")])
def test_two_streams_with_a_workspace_each(op, kind):
    p = Problem(op, kind, 40, 1024, 640, ranks=(16, 40, 9), seed=10)
    p.call()
    torch.cuda.synchronize()
    ref = p.y.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.full_like(p.y, SENTINEL) for _ in range(2)]
    wss = [torch.empty_like(p.ws) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, y, ws in zip(streams, ys, wss):
            p.call(stream=s, y=y, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ref) and torch.equal(ys[1], ref)
    p.close()


@pytest.mark.parametrize("op,kind,n", [("gemm", "int4z", 1), ("gemm", "int4", 200), ("glu", "bf16", 17), ("glu", "table", 64),
                                       ("glu", "fp8", 300)])
def test_captured_and_replayed(op, kind, n):
    """Kernels alone are enqueued: a captured call replays to the eager result, also on new x and
    ids written between the replays."""
    p = Problem(op, kind, n, 512, 320, ranks=(16, 40, 9), seed=11)
    p.call()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        p.call()
    for rep in range(3):
        p.x[:, :512].copy_(torch.randn(n, 512, device="cuda"))
        p.ids.copy_(torch.randint(-1, 3, (n,), device="cuda", dtype=torch.int32))
        eager = torch.full_like(p.y, SENTINEL)
        p.call(y=eager)
        p.y.fill_(SENTINEL)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y, eager), rep
    p.close()


@pytest.mark.parametrize("n", [40, 300])
def test_rows_far_apart(n):
    """Offsets of x and y past 2^31 elements: 64-bit addressing."""
    ld = 1 << 22
    rows = 520 if n == 300 else 40
    p = Problem("gemm", "int4", n, 256, 128, ranks=(16, 3), seed=12)
    big = torch.zeros(n * ld if n == 300 else 60 * ld, dtype=torch.bfloat16, device="cuda")
    x = big.view(-1, ld)[:n]
    x[:, :256].copy_(p.x)
    y = torch.full((600 * ld if n == 300 else 60 * ld,), SENTINEL, dtype=torch.bfloat16, device="cuda").view(-1, ld)[:n]
    sgr.lora_fused_gemm_w4(p.pool, 0, x, ld, p.wdev[0], p.ids, n, y, ld, p.ws)
    torch.cuda.synchronize()
    p.call()
    torch.cuda.synchronize()
    assert rows and torch.equal(y[:, :128], p.y[:n, :128])
    assert bool((y[:, 128:1024] == SENTINEL).all())
    p.close()


@pytest.mark.parametrize("n", [1, 48, 290])
def test_feed_forward_block(n):
    """Gate and up, the activation, the product and the down projection, all from 4-bit weights
    under adapters, as a layer runs them; the reference takes h as the call rounded it."""
    up = Problem("glu", "int4z", n, 256, 512, ranks=(16, 8, 30), seed=13, act="silu")
    up.call()
    up.check()
    h = up.y[:n].contiguous()
    down = Problem("gemm", "int4", n, 512, 256, group=128, ranks=(16, 8, 30), ids=up.ids64, seed=14,
                   x=h.double().cpu().numpy())
    down.x = h
    down.call()
    down.check()
    up.close()
    down.close()


def test_refusals():
    """Every refusal leaves y alone."""
    p = Problem("gemm", "int4", 8, 256, 128, group=64, ranks=(16,), seed=15)
    g = Problem("glu", "bf16", 8, 256, 128, ranks=(16,), seed=16)
    w = p.wdev[0]

    def w4(**kw):
        f = {k: getattr(w, k) for k, _ in sgr.lora_w4._fields_}
        f.update(kw)
        return sgr.lora_w4(*[f[k] for k, _ in sgr.lora_w4._fields_])

    def gemm(w4s=w, module=0, x=p.x.data_ptr(), ld_x=256, n=8, y=p.y.data_ptr(), ld_y=128, ws=p.ws.data_ptr(),
             ws_bytes=p.ws.numel() * 4):
        sgr.lora_fused_gemm_w4(p.pool, module, x, ld_x, w4s, p.ids, n, y, ld_y, ws, ws_bytes)

    def glu(mg=0, mu=1, act=0, wg=g.wdev[0].data_ptr(), wu=g.wdev[1].data_ptr(), ld_w=256, ws_bytes=g.ws.numel() * 4):
        sgr.lora_fused_glu(g.pool, mg, mu, g.x, 256, wg, wu, ld_w, g.ids, 8, act, g.y, 128, g.ws.data_ptr(), ws_bytes)

    cases = [
        (gemm, dict(module=2), -1), (gemm, dict(module=-1), -1), (gemm, dict(n=-1), -1),
        (gemm, dict(x=None), -1), (gemm, dict(y=None), -1), (gemm, dict(x=p.x.data_ptr() + 8), -1),
        (gemm, dict(ld_x=248), -1), (gemm, dict(ld_x=260), -1), (gemm, dict(ld_x=(1 << 22) + 8), -2),
        (gemm, dict(y=p.y.data_ptr() + 4), -1), (gemm, dict(ld_y=124), -1), (gemm, dict(ld_y=130), -1),
        (gemm, dict(ws_bytes=p.ws.numel() * 4 - 4), -9), (gemm, dict(ws=None, ws_bytes=0), -9),
        (gemm, dict(ws=p.ws.data_ptr() + 4), -1), (gemm, dict(ws=None), -1),
        (gemm, dict(w4s=w4(codes=None)), -1), (gemm, dict(w4s=w4(codes=w.codes + 8)), -1),
        (gemm, dict(w4s=w4(ld_codes=112)), -1), (gemm, dict(w4s=w4(ld_codes=136)), -1),
        (gemm, dict(w4s=w4(ld_codes=1 << 24)), -2),
        (gemm, dict(w4s=w4(scale=None)), -1), (gemm, dict(w4s=w4(scale=w.scale + 4)), -1),
        (gemm, dict(w4s=w4(ld_scale=124)), -1), (gemm, dict(w4s=w4(ld_scale=130)), -1),
        (gemm, dict(w4s=w4(group=16)), -1), (gemm, dict(w4s=w4(group=0)), -1), (gemm, dict(w4s=w4(group=256)), -1),
        (gemm, dict(w4s=w4(zero=w.scale, table=w.scale)), -1), (gemm, dict(w4s=w4(zero=w.scale + 2)), -1),
        (gemm, dict(w4s=w4(table=w.scale + 2)), -1),
        (glu, dict(mg=-1), -1), (glu, dict(mu=2), -1), (glu, dict(act=3), -1), (glu, dict(act=-1), -1),
        (glu, dict(wg=None), -1), (glu, dict(wu=None), -1), (glu, dict(wu=g.wdev[1].data_ptr() + 2), -1),
        (glu, dict(ld_w=248), -1), (glu, dict(ld_w=260), -1), (glu, dict(ld_w=1 << 23), -2), (glu, dict(ld_w=-8), -1),
        (glu, dict(ws_bytes=64), -9),
    ]
    for fn, kw, code in cases:
        with pytest.raises(sgr.LoraError) as ei:
            fn(**kw)
        assert ei.value.status == code, (fn.__name__, kw, ei.value.status)
    torch.cuda.synchronize()
    assert bool((p.y == SENTINEL).all()) and bool((g.y == SENTINEL).all())
    p.close()
    g.close()


def test_refusals_of_pools_and_pairs():
    """A group that does not divide h_in, widths that differ, unlike 4-bit pairs, an fp32 pool, too
    many pages to a rank row."""
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    w = sgr.lora_w4(t.data_ptr(), 512, t.data_ptr(), None, 512, None, 128)

    def status(fn):
        with pytest.raises(sgr.LoraError) as ei:
            fn()
        return ei.value.status

    pool = sgr.lora_pool_create(0, sgr.LORA_BF16, 64, 64, 2, 4, [192, 192, 128, 64 * 33], [128, 64, 128, 64], 4)
    assert status(lambda: sgr.lora_fused_gemm_w4(pool, 0, t, 192, w, None, 1, t, 128)) == -2
    assert status(lambda: sgr.lora_fused_glu(pool, 0, 1, t, 192, t, t, 192, None, 1, 0, t, 128)) == -2
    assert status(lambda: sgr.lora_fused_glu(pool, 0, 2, t, 192, t, t, 192, None, 1, 0, t, 128)) == -2
    assert status(lambda: sgr.lora_fused_glu(pool, 3, 3, t, 64 * 33, t, t, 64 * 33, None, 1, 0, t, 64)) == -2
    for other in (sgr.lora_w4(t.data_ptr(), 512, t.data_ptr(), None, 512, None, 64),
                  sgr.lora_w4(t.data_ptr(), 528, t.data_ptr(), None, 512, None, 128),
                  sgr.lora_w4(t.data_ptr(), 512, t.data_ptr(), None, 512, t.data_ptr(), 128)):
        assert status(lambda: sgr.lora_fused_glu_w4(pool, 2, 2, t, 128, w, other, None, 1, 0, t, 128)) == -2
    assert status(lambda: sgr.lora_fused_glu_fp8w(pool, 2, 2, t, 128, t, t, 128, t, None, None, 1, 0, t, 128)) == -1
    assert sgr.lora_fused_workspace_bytes(pool, 9, 1, 1) == 0 and sgr.lora_fused_workspace_bytes(pool, 0, 3, 1) == 0
    f32 = sgr.lora_pool_create(0, sgr.LORA_F32, 64, 64, 2, 1, [128], [128], 4)
    assert status(lambda: sgr.lora_fused_gemm_w4(f32, 0, t, 128, w, None, 1, t, 128)) == -6
    sgr.lora_pool_destroy(pool)
    sgr.lora_pool_destroy(f32)


@pytest.mark.parametrize("n", [(1 << 28) + 256, (1 << 31) - 1])
def test_batches_past_a_launch(n):
    """Refused before anything is launched; the workspace query counts them all the same."""
    p = Problem("gemm", "int4", 4, 256, 64, group=64, ranks=(16,), seed=51)
    g = Problem("glu", "bf16", 4, 256, 64, ranks=(16,), seed=52)
    assert sgr.lora_fused_workspace_bytes(p.pool, 0, 1, n) == 4 * n * 64
    for q in (p, g):
        with pytest.raises(sgr.LoraError) as ei:
            q.call(n=n)
        assert ei.value.status == -2
        torch.cuda.synchronize()
        assert bool((q.y == SENTINEL).all())
        q.close()
