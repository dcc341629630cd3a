"""An adapter whose weights hold an infinity or NaN spoils the outputs of its own
tokens and of no others, whichever way the base products and the fused passes
take: the tokens of other adapters and those without one keep their bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import segmented_gathered_rank_amd as sgr  # noqa: E402
from base_util import Problem, bf16  # noqa: E402

BITS = {"bf16": 16, "fp8": 8}
FORMS = [("gemm", "int4", 64), ("gemm", "table", 32), ("glu", "bf16", 0), ("glu", "fp8", 0), ("glu", "int4z", 32)]
BAD_SLOT = 1


def _reload(p, which, bad):
    """Slot BAD_SLOT again, with `bad` in some places of A or B of its last module."""
    sgr.lora_pool_evict(p.pool, BAD_SLOT)
    for m in range(2):
        sc, a, b = (np.array(v) for v in p.adapters[m][BAD_SLOT])
        if m == p.np - 1:
            (a if which == "a" else b)[1, 5::40] = bad
        sgr.lora_pool_load(p.pool, BAD_SLOT, m, a.shape[0], bf16(a), bf16(b), float(sc))


def _spoiled(p, call, which, bad):
    call()
    torch.cuda.synchronize()
    clean = p.y.clone()
    assert torch.isfinite(clean[:p.n, :p.h_out]).all()
    _reload(p, which, bad)
    p.y.zero_()
    call()
    torch.cuda.synchronize()
    own = p.ids.cpu().numpy() == BAD_SLOT
    assert own.any() and not own.all()
    assert torch.equal(p.y[:p.n][~own].view(torch.int16), clean[:p.n][~own].view(torch.int16))
    y = p.y[:p.n][own][:, :p.h_out]
    if which == "a":
        assert not torch.isfinite(y).any()
    else:
        hit = torch.zeros(p.h_out, dtype=torch.bool, device="cuda")
        hit[5::40] = True
        assert not torch.isfinite(y[:, hit]).any() and torch.isfinite(y[:, ~hit]).all()
    p.close()


@pytest.mark.parametrize("op,kind,group", FORMS, ids=[f"{o}-{k}-{g}" for o, k, g in FORMS])
@pytest.mark.parametrize("way", ["rows", "tiles"])
@pytest.mark.parametrize("which", ["a", "b"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_base_products(op, kind, group, way, which, bad):
    n, h_out = (50, 320) if way == "rows" else (300, 15040 if op == "gemm" else 8000)
    p = Problem(op, kind, n, 256, h_out, group=group or 64, ranks=(16, 11, 4), seed=33)
    tiles = sgr.lora_fused_tile_tokens(p.pool, 0, p.np, BITS.get(kind, 4), n, True)
    assert tiles == (n if way == "tiles" else 0)
    _spoiled(p, p.call, which, bad)


@pytest.mark.parametrize("ranks", [(16, 11), (16, 11, 4, 64)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("which", ["a", "b"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_fused_passes(ranks, kind, which, bad):
    """lora_fused_gemm and lora_fused_gemm_fp8w, with units that ride along and units of further passes."""
    p = Problem("glu", kind, 300, 256, 320, ranks=ranks, seed=34)
    p.np = 1

    def call():
        if kind == "bf16":
            sgr.lora_fused_gemm(p.pool, 0, p.x, p.ld_x, p.wdev[0], p.ld_w, p.ids, p.n, p.y, p.ld_y)
        else:
            sgr.lora_fused_gemm_fp8w(p.pool, 0, p.x, p.ld_x, p.wdev[0][0], p.ld_w, p.wdev[0][1], p.ids, p.n, p.y,
                                     p.ld_y)

    _spoiled(p, call, which, bad)
