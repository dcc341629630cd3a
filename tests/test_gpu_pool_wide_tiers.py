"""Adapter tiers over a pool whose entries span more than 1024 pages: adapters come
and go through fewer slots than adapters, and the fused pass reads what is there."""
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
from segmented_gathered_rank_amd.harness import from_device, to_device  # noqa: E402


def test_tiers_serve_a_wide_pool():
    wl = W.tier_batches(seed=29)
    bsz, mod = wl.notes["batch"], wl.modules[0]
    rng = np.random.default_rng(6)
    n_slots, host_slots, wide_out = 4, 6, 64 * 18
    # a second module of 64 x 1152 in pages of 64: with a cap of 64 ranks its entries span 64 * 19 pages
    per = 64 * max((mod.h_in + mod.h_out) // 64, 19)
    pool = sgr.lora_pool_create(0, sgr.LORA_BF16, 64, n_slots * 2 * per, n_slots, 2, [mod.h_in, 64],
                                [mod.h_out, wide_out], 64)
    wide = {a: (int(r), 0.25, rng.integers(0, 1 << 15, (r, 64), dtype=np.uint16) & 0xBF7F,
                rng.integers(0, 1 << 15, (r, wide_out), dtype=np.uint16) & 0xBF7F)
            for a, r in ((a, rng.choice([1, 17, 64])) for a in range(wl.n_slots))}
    tiers = sgr.lora_tiers_create(n_slots, host_slots)

    def fetch(adapter, module):
        if module == 1:
            return wide[adapter]
        a = wl.adapters[adapter][0]
        return None if a is None else (a[0], a[1], a[2], a[3])

    dev = torch.device("cuda", 0)
    x = to_device(wl.x[0], "bf16", dev)
    w = torch.zeros(mod.h_out, mod.h_in, dtype=torch.bfloat16, device=dev)
    y = torch.zeros(wl.n_tokens, mod.h_out, dtype=torch.bfloat16, device=dev)
    for b in range(wl.n_tokens // bsz):
        ids = wl.ids[b * bsz:(b + 1) * bsz]
        req = ids[ids >= 0]
        slots = sgr.lora_tiers_acquire(tiers, pool, req, fetch)
        tok = np.full(bsz, -1, np.int32)
        tok[ids >= 0] = slots
        d_ids = torch.from_numpy(tok).to(dev)
        sgr.lora_fused_gemm(pool, 0, x[b * bsz:], mod.h_in, w, mod.h_in, d_ids, bsz, y[b * bsz:], mod.h_out)
        for a, s in {int(a): int(s) for a, s in zip(req, slots)}.items():
            rank, scale, wa, wb = wide[a]
            ra, rb = np.zeros_like(wa), np.zeros_like(wb)
            got = sgr.lora_pool_read(pool, s, 1, ra, rb)
            assert got[0] == rank and got[1] == scale and np.array_equal(ra, wa) and np.array_equal(rb, wb)
    torch.cuda.synchronize()
    ref = lo.lora_delta(wl, 0, list(range(wl.n_tokens)))
    assert_close(lo.decode(from_device(y), "bf16"), ref, "bf16", "tiers, wide pool")
    assert sgr.lora_pool_stats(pool)["evicts"] > 0
    sgr.lora_tiers_destroy(tiers)
    sgr.lora_pool_destroy(pool)
