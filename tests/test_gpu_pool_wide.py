"""A pool whose entries span more than 1024 pages: loads and reads back, serves
lora_fused_gemm, and every apply call that keeps page ids in a 1024-word table
refuses it."""
import numpy as np
import pytest

import workloads as W
from oracle import lora_oracle as lo

from gpu_util import assert_close

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import segmented_gathered_rank_amd as sgr  # noqa: E402
from segmented_gathered_rank_amd.harness import DeviceWorkload, from_device  # noqa: E402


def _wide():
    """fused_tiles with its widths kept (320 -> 384, pages of 64) and a second module of 64 x 1152
    whose entries, at rank 64, span 64 * 19 = 1216 pages."""
    wl = W.fused_tiles(seed=23)
    pool = sgr.lora_pool_create(0, sgr.LORA_BF16, 64, wl.pages_needed() + 2048, wl.n_slots, 2, [320, 64], [384, 1152],
                                64)
    for s, row in enumerate(wl.adapters):
        if row[0] is not None:
            rank, scale, a, b = row[0]
            sgr.lora_pool_load(pool, s, 0, rank, np.ascontiguousarray(a), np.ascontiguousarray(b), scale)
    return wl, pool


def test_wide_entries_load_and_read_back():
    wl, pool = _wide()
    rng = np.random.default_rng(5)
    a = rng.integers(0, 1 << 16, (64, 64), dtype=np.uint16)
    b = rng.integers(0, 1 << 16, (64, 1152), dtype=np.uint16)
    sgr.lora_pool_load(pool, 3, 1, 64, a, b, 0.5)
    ra, rb = np.zeros_like(a), np.zeros_like(b)
    rank, scale, pages = sgr.lora_pool_read(pool, 3, 1, ra, rb, max_pages=1216)
    assert rank == 64 and scale == 0.5 and len(set(pages)) == 1216
    assert np.array_equal(ra, a) and np.array_equal(rb, b)
    sgr.lora_pool_destroy(pool)


def test_wide_pool_serves_the_fused_pass_and_refuses_the_apply_calls():
    wl, pool = _wide()
    dw = DeviceWorkload(wl)
    dw.upload_weights()
    n = wl.n_tokens
    y = dw.y_of(0)
    sgr.lora_fused_gemm(pool, 0, dw._xp(0), 320, dw.wT[0], 320, dw.ids, n, y, 384)
    torch.cuda.synchronize()
    got = lo.decode(from_device(y), "bf16")
    assert_close(got, lo.lora_forward(wl, 0, list(range(n))), "bf16", "wide pool, fused pass")
    before = y.clone()
    x, t = dw._xp(0), dw.t
    calls = [
        lambda: sgr.lora_shrink(pool, 0, 1, x, 320, 0, dw.seg, t, dw.ld_t, 0),
        lambda: sgr.lora_shrink_noalloc(pool, 0, 1, x, 320, 0, dw.seg, t, dw.ld_t, 0),
        lambda: sgr.lora_expand(pool, 0, 1, t, dw.ld_t, 0, dw.seg, y, 384, 0, sgr.LORA_BF16),
        lambda: sgr.lora_apply_sgmv(pool, 0, 1, x, 320, 0, dw.seg, t, dw.ld_t, 0, y, 384, 0, sgr.LORA_BF16),
        lambda: sgr.lora_apply_bgmv(pool, 0, 1, x, 320, 0, dw.seg, y, 384, 0, sgr.LORA_BF16),
        lambda: sgr.lora_apply_bgmv_ids(pool, 0, 1, x, 320, 0, dw.ids, 8, y, 384, 0, sgr.LORA_BF16),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(sgr.LoraError) as ei:
            call()
        assert ei.value.status == -2, k
    torch.cuda.synchronize()
    assert torch.equal(y, before)
    dw.close()
    sgr.lora_pool_destroy(pool)


def test_pool_refuses_entries_above_the_cap():
    with pytest.raises(sgr.LoraError) as ei:
        sgr.lora_pool_create(0, sgr.LORA_BF16, 64, 64, 1, 1, [64], [64 * 128], 64)   # 64 * 129 pages
    assert ei.value.status == -2
