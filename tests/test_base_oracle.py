"""Pins of the fp64 definitions of the 4-bit base weights and the gated product,
and the host-side refusals that need no GPU."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import base_oracle as bo


def test_unpack_order_low_nibble_first():
    codes = np.array([[0x21, 0x43], [0xF0, 0x8E]], np.uint8)
    assert bo.unpack_w4(codes, 4).tolist() == [[1, 2, 3, 4], [0, 15, 14, 8]]


@pytest.mark.parametrize("form", ["plain", "zero", "table"])
def test_widen_w4_against_rationals(form):
    rng = np.random.default_rng(3)
    h_in, h_out, group = 64, 5, 32
    codes = rng.integers(0, 256, (h_out, h_in // 2), dtype=np.uint8)
    scale = rng.integers(-8, 9, (2, h_out)) / 16.0
    zero = rng.integers(0, 256, (2, h_out), dtype=np.uint8) if form == "zero" else None
    table = rng.integers(-64, 65, 16) / 32.0 if form == "table" else None
    w = bo.widen_w4(codes, scale, group, zero, table)
    for k in range(h_in):
        for c in range(h_out):
            q = int(codes[c, k // 2]) // (16 if k % 2 else 1) % 16
            v = Fraction(table[q]) if form == "table" else Fraction(q - (8 if zero is None else int(zero[k // group, c])))
            assert Fraction(w[k, c]) == Fraction(scale[k // group, c]) * v


def test_activations_closed_forms():
    v = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    for act in ("silu", "gelu", "gelu_tanh"):
        a = bo.activation(act, v)
        assert a[2] == 0 and abs(a[4] - 30) < 1e-11 and abs(a[0]) < 1e-11
        assert np.allclose(a[3] + bo.activation(act, -v[3:4])[0], a[3] + a[1])
        assert np.allclose(bo.activation(act, v) - bo.activation(act, -v), v)   # act(v) - act(-v) = v
    assert abs(bo.activation("silu", np.array([1.0]))[0] - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(bo.activation("gelu", np.array([1.0]))[0] - 0.8413447460685429) < 1e-15


def test_linear_merged_weights():
    rng = np.random.default_rng(4)
    x, w = rng.normal(size=(6, 8)), rng.normal(size=(8, 5))
    ad = [(2.0, rng.normal(size=(3, 8)), rng.normal(size=(3, 5))), None]
    ids = [0, -1, 1, 0, 2, 0]
    y, _ = bo.linear(x, w, ids, ad)
    merged = w + 2.0 * ad[0][1].T @ ad[0][2]
    for i, a in enumerate(ids):
        assert np.allclose(y[i], x[i] @ (merged if a == 0 else w), atol=1e-12)


def test_base_calls_refuse_a_null_pool():
    import segmented_gathered_rank_amd as sgr
    w = sgr.lora_w4(1 << 20, 64, 1 << 20, None, 64, None, 32)
    for call in (lambda: sgr.lora_fused_gemm_w4(0, 0, 16, 64, w, None, 1, 16, 64),
                 lambda: sgr.lora_fused_glu(0, 0, 1, 16, 64, 16, 16, 64, None, 1, sgr.LORA_ACT_SILU, 16, 64),
                 lambda: sgr.lora_fused_glu_fp8w(0, 0, 1, 16, 64, 16, 16, 64, 16, 16, None, 1, 0, 16, 64),
                 lambda: sgr.lora_fused_glu_w4(0, 0, 1, 16, 64, w, w, None, 1, 0, 16, 64)):
        with pytest.raises(sgr.LoraError) as ei:
            call()
        assert ei.value.status == -1
    assert sgr.lora_fused_workspace_bytes(0, 0, 1, 1) == 0
