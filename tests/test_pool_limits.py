"""Pool shapes that are refused before the device is touched (CPU)."""
import pytest

import segmented_gathered_rank_amd as sgr


def _status(dtype, h_out, h_in=64):
    with pytest.raises(sgr.LoraError) as ei:
        sgr.lora_pool_destroy(sgr.lora_pool_create(0, dtype, 64, 64, 1, 1, [h_in], [h_out], 64))
    return ei.value.status


def test_fp32_pools_of_wide_entries():
    """Only the fused passes read entries of more than 1024 pages, and those are bf16: an fp32 pool
    of such entries would be one that no call serves."""
    assert _status(sgr.LORA_F32, 64 * 16) == -2      # 64 * 17 pages


def test_wide_entries_of_many_pages_to_a_row():
    """The fused passes hold 32 pages of a row of A: wide entries with more would be no call's either."""
    assert _status(sgr.LORA_BF16, 64, h_in=64 * 33) == -2      # 64 * 34 pages


def test_entries_above_the_cap():
    assert _status(sgr.LORA_F32, 64 * 128) == -2 and _status(sgr.LORA_BF16, 64 * 128) == -2
