"""What a call of the 4-bit and gated products needs of a workspace, on both ways:
the least is accepted, 16 bytes less are refused with y and the workspace left
alone, and nothing behind the workspace is written."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import segmented_gathered_rank_amd as sgr  # noqa: E402
from base_util import SENTINEL, Problem  # noqa: E402

BITS = {"bf16": 16, "fp8": 8}
GUARD = -55.0
# n, h_in, h_out by operator, the splits of h_in on tiles (64 tokens to a workgroup of at least 256 k)
SHAPES = {
    "rows, one block": (7, 2048, 256), "rows": (40, 2048, 256), "rows, chunks": (150, 1024, 320),
    "tiles": (300, 256, None), "tiles, split": (300, 1024, None),
}


def _problem(op, kind, shape, ids="random"):
    n, h_in, h_out = SHAPES[shape]
    if h_out is None:
        h_out = 16064 if op == "gemm" else 8064
        if h_in == 1024:
            h_out *= 2
    page = 128 if shape == "tiles, split" else 64
    p = Problem(op, kind, n, h_in, h_out, page=page, group=64, ranks=(16, 5), ids=ids, seed=61, w_scale=0.02)
    tiles = sgr.lora_fused_tile_tokens(p.pool, 0, p.np, BITS.get(kind, 4), n, p.ids is not None)
    if ids == "random":
        assert tiles == (n if shape.startswith("tiles") else 0)
    # fp32: base sums of one split and 64 of t for each token and projection, or t alone from each split
    least = 4 * p.np * n * ((h_out + 64) if tiles == 0 else 64 * (h_in // 256))
    return p, least


def _with(p, nbytes):
    """The call with nbytes of a guarded buffer; returns whether the guard is whole."""
    buf = torch.full((nbytes // 4 + 4096,), GUARD, device="cuda")
    ws = buf[2048:2048 + nbytes // 4]
    p.y.fill_(SENTINEL)
    torch.cuda.synchronize()
    try:
        p.call(ws=ws)
    finally:
        torch.cuda.synchronize()
        assert bool((buf[:2048] == GUARD).all()) and bool((buf[2048 + nbytes // 4:] == GUARD).all()), "wrote past ws"
    return ws


@pytest.mark.parametrize("op,kind", [("gemm", "int4z"), ("gemm", "table"), ("glu", "bf16"), ("glu", "fp8")])
@pytest.mark.parametrize("shape", SHAPES)
def test_least_workspace(op, kind, shape):
    p, least = _problem(op, kind, shape)
    full = sgr.lora_fused_workspace_bytes(p.pool, 0, p.np, p.n)
    assert least <= full and least % 16 == 0
    for nbytes in sorted({least, (least + full) // 2 // 16 * 16, full}):
        _with(p, nbytes)
        p.check(what=f"{nbytes} of {full} bytes")
    for nbytes in (least - 16, 16):
        with pytest.raises(sgr.LoraError) as ei:
            _with(p, nbytes)
        assert ei.value.status == -9
        assert bool((p.y == SENTINEL).all())
    p.close()


@pytest.mark.parametrize("op,kind", [("gemm", "int4z"), ("glu", "bf16")])
@pytest.mark.parametrize("shape", SHAPES)
def test_any_workspace_without_ids(op, kind, shape):
    p, _ = _problem(op, kind, shape, ids="null")
    full = sgr.lora_fused_workspace_bytes(p.pool, 0, p.np, p.n)
    for nbytes in (16, full // 3 // 16 * 16, full):
        _with(p, nbytes)
        p.check(what=f"{nbytes} of {full} bytes")
    p.ws = None
    p.y.fill_(SENTINEL)
    p.call()
    p.check(what="none")
    p.close()
