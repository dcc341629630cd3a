"""The 4-bit and gated base products on tiles (long batches): every weight kind,
group and activation with and without ids, at shapes for which
lora_fused_tile_tokens says that tiles are taken (wide h_out and few k: little
work for the oracle, and the costs choose tiles), and which end inside a tile on
every side.  Each test asserts the way it takes.

Tiles multiply x by the exact v of a 4-bit weight, so the bound counts |s v| and
not, as on the other way, the codes and zero points apart."""
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
         ("gemm", "table", 128), ("glu", "bf16", 0), ("glu", "fp8", 0), ("glu", "int4", 32), ("glu", "int4", 64),
         ("glu", "int4", 128), ("glu", "int4z", 32), ("glu", "int4z", 64), ("glu", "int4z", 128),
         ("glu", "table", 32), ("glu", "table", 64), ("glu", "table", 128)]
FORM_IDS = [f"{o}-{k}-{g}" for o, k, g in FORMS]
SOME = [("gemm", "int4", 64), ("gemm", "int4z", 32), ("gemm", "table", 128), ("glu", "bf16", 0), ("glu", "fp8", 0),
        ("glu", "int4z", 128), ("glu", "table", 32)]
SOME_IDS = [f"{o}-{k}-{g}" for o, k, g in SOME]
BITS = {"bf16": 16, "fp8": 8}


def _tiled(op, kind, n, h_in, h_out, group=64, **kw):
    """A problem all of whose tokens take tiles.  h_out: of one projection (gemm) or of the gate's two."""
    p = Problem(op, kind, n, h_in, h_out, group=group or 64, **kw)
    with_ids = p.ids is not None
    tiles = sgr.lora_fused_tile_tokens(p.pool, 0, p.np, BITS.get(kind, 4), n, with_ids)
    assert tiles == n
    p.wabs = [np.abs(w) for w in p.w64]
    return p


def _run(*a, **kw):
    p = _tiled(*a, **kw)
    p.call()
    worst = p.check(what=str(a))
    p.close()
    return worst


def _wide(op):
    return 15040 if op == "gemm" else 8000     # end 192 into 256 columns and 64 into 128


@pytest.mark.parametrize("op,kind,group", FORMS, ids=FORM_IDS)
def test_with_adapters(op, kind, group):
    """Neighbours of different adapters, one of them not loaded, and tokens without one."""
    _run(op, kind, 300, 256, _wide(op), group, ranks=(16, 3, 1, 0, 9), seed=group + 1)


@pytest.mark.parametrize("op,kind,group", FORMS, ids=FORM_IDS)
def test_without_ids(op, kind, group):
    _run(op, kind, 300, 256, 25024 if op == "gemm" else 12608, group, ranks=(4,), ids="null", act="gelu",
         seed=group + 2)


@pytest.mark.parametrize("op,kind,group", FORMS, ids=FORM_IDS)
@pytest.mark.parametrize("long", [False, True])
def test_padded_rows_and_odd_widths(op, kind, group, long):
    """One step of k (two for groups of 128) and an odd number of them; rows padded by NaN (x, bf16
    weights, fp8 codes) and by other codes; zero points up to 255."""
    h_in = (640 if group == 128 else 448) if long else (128 if group == 128 else 64)
    _run(op, kind, 300, h_in, 18112 if op == "gemm" else 9152, group, ranks=(8, 13), act="gelu_tanh", pads=3,
         seed=h_in)


@pytest.mark.parametrize("op,kind,group", SOME, ids=SOME_IDS)
@pytest.mark.parametrize("ids", ["none", "bad", "runs", "one"])
def test_kinds_of_ids(op, kind, group, ids):
    _run(op, kind, 300, 256, _wide(op), group, ranks=(16, 3, 5), ids=ids, act="gelu", seed=17)


@pytest.mark.parametrize("op,kind,group", [("gemm", "int4z", 64), ("gemm", "table", 32), ("glu", "bf16", 0),
                                           ("glu", "fp8", 0), ("glu", "int4", 64)])
def test_ranks_to_64(op, kind, group):
    """Up to 14 units of 16 rank rows to a projection: several passes of the shrink, several pairs of
    the expand; pages that end inside a tile."""
    n, h_out = (600, 16320) if op == "gemm" else (1000, 8000)
    _run(op, kind, n, 320, h_out, group, page=320, ranks=(64, 33, 16, 0, 17), seed=18)


@pytest.mark.parametrize("op,kind,h_in,h_out", [("gemm", "int4", 256, 16064), ("glu", "bf16", 512, 8000)])
def test_256_adapters_in_a_tile(op, kind, h_in, h_out):
    _run(op, kind, 1000, h_in, h_out, ranks=(4,) * 600, ids=np.arange(1000)[::-1] % 600, seed=19)


def test_unlike_neighbours_of_40_adapters():
    _run("glu", "table", 1000, 1280, 8000, 32, page=320, ranks=(8, 16, 32, 64) * 10, ids=np.arange(1000) * 7 % 40,
         seed=20)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4", "table"])
def test_adapter_on_one_projection_only(kind):
    _run("glu", kind, 300, 256, 8000, ranks=(16, 16, 16, 16), load=lambda s, p: (s >> p) & 1 == 1, seed=21)


def test_one_module_for_both_projections():
    p = _tiled("glu", "bf16", 300, 256, 8000, ranks=(16, 7), seed=22)
    for modules in ((1, 1), (1, 0)):
        p.call(modules=modules)
        p.check(modules=modules)
    p.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4", "int4z", "table"])
@pytest.mark.parametrize("ids", ["random", "null"])
def test_many_row_tiles(kind, ids):
    """Seven row tiles: the gated pass takes four at a time and the last three."""
    _run("glu", kind, 1546, 128, 3904 if ids == "random" else 8000, 32, ranks=(16, 3, 5), ids=ids, seed=23)


@pytest.mark.parametrize("op,kind,group", SOME, ids=SOME_IDS)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_rows_stay_in_their_rows(op, kind, group, bad):
    n, at = 300, 271
    x = np.random.default_rng(3).normal(size=(n, 256))
    clean = _tiled(op, kind, n, 256, _wide(op), group, ranks=(16, 8), seed=24, x=x)
    x2 = x.copy()
    x2[at, 100] = bad
    p = _tiled(op, kind, n, 256, _wide(op), group, ranks=(16, 8), seed=24, x=x2)
    clean.call()
    p.call()
    torch.cuda.synchronize()
    keep = np.arange(n) != at
    assert torch.equal(p.y[:n][keep].view(torch.int16), clean.y[:n][keep].view(torch.int16))
    assert not torch.isfinite(p.y[at, :p.h_out]).all()
    clean.close()
    p.close()


@pytest.mark.parametrize("op,kind,group", SOME, ids=SOME_IDS)
def test_same_bits_every_time_and_on_another_stream(op, kind, group):
    p = _tiled(op, kind, 300, 256, _wide(op), group, ranks=(16, 9), seed=25)
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


@pytest.mark.parametrize("op,kind,group", SOME, ids=SOME_IDS)
def test_captured_and_replayed(op, kind, group):
    p = _tiled(op, kind, 300, 256, _wide(op), group, ranks=(16, 3, 9), seed=26)
    p.call()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        p.call()
    for rep in range(3):
        p.x[:, :256].copy_(torch.randn(300, 256, device="cuda"))
        p.ids.copy_(torch.randint(-1, 3, (300,), device="cuda", dtype=torch.int32))
        eager = torch.full_like(p.y, SENTINEL)
        p.call(y=eager)
        p.y.fill_(SENTINEL)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y, eager), rep
    p.close()


def test_rows_far_apart():
    """Offsets of x and y past 2^31 bytes and 2^30 elements within a launch."""
    n, ld = 300, 1 << 22
    p = _tiled("gemm", "int4z", n, 256, 15040, 32, ranks=(16, 3), seed=27)
    x = torch.zeros(n * ld, dtype=torch.bfloat16, device="cuda").view(n, ld)
    x[:, :256].copy_(p.x)
    y = torch.full((n * ld,), SENTINEL, dtype=torch.bfloat16, device="cuda").view(n, ld)
    sgr.lora_fused_gemm_w4(p.pool, 0, x, ld, p.wdev[0], p.ids, n, y, ld, p.ws)
    p.call()
    torch.cuda.synchronize()
    assert torch.equal(y[:, :15040], p.y[:n, :15040])
    assert bool((y[:, 15040:20000] == SENTINEL).all())
    p.check()
    p.close()


@pytest.mark.parametrize("op,kind,group", [("gemm", "int4z", 64), ("glu", "bf16", 0), ("glu", "int4z", 32)])
def test_a_rest_on_rows(op, kind, group):
    """32 row tiles fill the GPU once and the 40 tokens behind them take the other way; the oracle at
    the tokens around the seam and some others."""
    n, h_out = 32 * 256 + 40, 2048 if op == "gemm" else 1024
    p = Problem(op, kind, n, 2048, h_out, page=256, group=group or 64, ranks=(16, 5), ids="runs", seed=28,
                w_scale=0.02)
    assert sgr.lora_fused_tile_tokens(p.pool, 0, p.np, BITS.get(kind, 4), n, True) == n - 40
    p.call()
    torch.cuda.synchronize()
    got = p.y.double().cpu().numpy()
    assert np.all(got[n:] == SENTINEL)
    toks = np.unique(np.concatenate([np.arange(n - 60, n), np.random.default_rng(1).integers(0, n, 150)]))
    x, ids = p.x64, p.ids64
    p.x64, p.ids64 = x[toks], ids[toks]
    v, bound = p.reference()
    assert np.all(np.abs(got[toks] - v) <= bound)
    p.close()


def test_tile_tokens_arguments():
    p = Problem("gemm", "int4", 4, 256, 64, group=64, ranks=(16,), seed=29)
    ask = lambda module=0, n_proj=1, bits=4, n=1000, ids=True: sgr.lora_fused_tile_tokens(p.pool, module, n_proj, bits,
                                                                                          n, ids)
    for kw in (dict(module=-1), dict(module=2), dict(n_proj=0), dict(n_proj=3), dict(bits=5), dict(n=-1)):
        assert ask(**kw) == -1
    assert ask(n=0) == 0 and ask(n=64) == 0 and 0 <= ask() <= 1000
    p.close()
