"""fp64 definitions of the base products with quantized weights and of the gated
feed-forward product.  Plain numpy; shares no code with the HIP side.

Every function takes arrays of exact values (float64) or integer codes.
"""
from __future__ import annotations

import math

import numpy as np

from . import lora_oracle as lo

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def unpack_w4(codes: np.ndarray, h_in: int) -> np.ndarray:
    """[h_out][>= h_in / 2] bytes -> [h_out][h_in] codes 0..15; k even in a byte's low four bits."""
    out = np.empty((codes.shape[0], h_in), np.int64)
    for k in range(h_in):
        out[:, k] = (codes[:, k // 2] >> (4 * (k % 2))) & 15
    return out


def widen_w4(codes, scale, group, zero=None, table=None) -> np.ndarray:
    """W [h_in][h_out]: scale[k / group][c] * v(code); scale, zero [h_in / group][h_out], table [16]."""
    n_g, h_out = scale.shape
    q = unpack_w4(codes, n_g * group).T
    g = np.arange(n_g * group) // group
    if table is not None:
        v = np.asarray(table, np.float64)[q]
    else:
        v = q - (8.0 if zero is None else zero.astype(np.float64)[g])
    return scale.astype(np.float64)[g] * v


def widen_fp8(codes, scale) -> np.ndarray:
    """W [h_in][h_out] from [h_out][h_in] E4M3 codes and a scale per output column."""
    return (lo.decode_e4m3(codes) * scale.astype(np.float64)[:, None]).T


def linear(x, w, ids=None, adapters=None):
    """x W + s (x A^T) B per token.  adapters[slot] = (scale, A [r][h_in], B [r][h_out]) or None.
    Returns (y, S): S bounds the sum of the absolute products behind each y, for error bounds."""
    y = x @ w
    s = np.abs(x) @ np.abs(w)
    if ids is not None:
        for i, a in enumerate(ids):
            if 0 <= a < len(adapters) and adapters[a] is not None:
                sc, A, B = adapters[a]
                y[i] += sc * ((x[i] @ A.T) @ B)
                s[i] += abs(sc) * ((np.abs(x[i]) @ np.abs(A).T) @ np.abs(B))
    return y, s


def activation(act: str, v: np.ndarray) -> np.ndarray:
    if act == "silu":
        return v / (1.0 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    assert act == "gelu_tanh"
    return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))


def gated(act: str, g: np.ndarray, u: np.ndarray) -> np.ndarray:
    return activation(act, g) * u
