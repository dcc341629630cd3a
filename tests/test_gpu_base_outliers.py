"""Outliers of x under weights of value zero (codes equal to the zero point): exact
on tiles, and on rows off by the roundings that the header gives for sums of q x
and z x formed apart."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import segmented_gathered_rank_amd as sgr  # noqa: E402
from base_util import Problem  # noqa: E402


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,h_out", [(5, 192), (40, 192), (300, 15040)])
def test_outliers_under_zero_weights(group, n, h_out):
    h_in, at = 256, np.arange(6, 256, 32)            # an even k in every group
    x = np.random.default_rng(5).normal(size=(n, h_in))
    x[:, at] = 3e4 * np.sign(x[:, at])
    p = Problem("gemm", "int4", n, h_in, h_out, group=group, ranks=(4,), ids="none", seed=71, x=x)
    tiles = sgr.lora_fused_tile_tokens(p.pool, 0, 1, 4, n, True)
    assert tiles == (n if n == 300 else 0)
    codes = p.wdev[0]._keep[0]
    codes[:, at // 2] = (codes[:, at // 2] & 0xF0) | 8
    # the bound's weights where the zero point joins after the product: |s v| + 2 |s| z; a row's |s| z is there already
    p.wabs[0][at] -= np.abs(p.w64[0][at])
    p.w64[0][at] = 0.0
    if tiles:
        p.wabs = [np.abs(w) for w in p.w64]
    p.call()
    p.check(what=f"group {group}, {n} tokens")
    p.close()
