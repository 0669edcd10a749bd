"""Oracle of the e4m3 quantizer, the residual RMS norm and the block-scaled
product (test infrastructure only; see the package docstring).

e4m3 has a sign, four exponent bits of bias 7 and three mantissa bits: code
magnitude c = 8 e + f stands for 2^(e - 7) (1 + f / 8), for e = 0 for 2^-6 f / 8,
and c = 127 for NaN; the largest value is 448.  Blocks are 1 or 128 rows by 128
columns; a block's scale is max(m, 1e-30) / 448 with m its largest magnitude.
"""
from __future__ import annotations

import numpy as np

GROUP = 128
AMAX_FLOOR = np.float32(1e-30)


def _table() -> np.ndarray:
    c = np.arange(128)
    e, f = c >> 3, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v[127] = np.nan
    return np.concatenate([v, -v])


VALUES = _table()
_MAGNITUDES = VALUES[:127]


def decode(codes: np.ndarray) -> np.ndarray:
    """e4m3 codes (uint8) -> float64 values."""
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 codes of values of at most 448 (ties to the even code)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(v, nan=0.0)), 448.0)
    hi = np.searchsorted(_MAGNITUDES, a, side="left")
    lo = np.maximum(hi - 1, 0)
    up, down = _MAGNITUDES[hi] - a, a - _MAGNITUDES[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.isnan(v), 127, c)
    return (c + 128 * np.signbit(v)).astype(np.uint8)


def block_amax(x: np.ndarray, block_rows: int) -> np.ndarray:
    rows, cols = x.shape
    out = np.empty((-(-rows // block_rows), cols // GROUP), dtype=x.dtype)
    for i in range(out.shape[0]):
        for g in range(out.shape[1]):
            out[i, g] = np.max(np.abs(x[i * block_rows:(i + 1) * block_rows, g * GROUP:(g + 1) * GROUP]))
    return out


def spread(per_block: np.ndarray, block_rows: int, rows: int) -> np.ndarray:
    """One value per block -> one per element."""
    return np.kron(per_block, np.ones((block_rows, GROUP), per_block.dtype))[:rows]


def quantize(x: np.ndarray, block_rows: int):
    """The quantizer step by step in float32: (codes, scales), bit for bit."""
    x = np.asarray(x, dtype=np.float32)
    m = np.maximum(block_amax(x, block_rows), AMAX_FLOOR)
    r = np.float32(448.0) / m
    codes = encode(x * spread(r, block_rows, x.shape[0]))
    return codes, m / np.float32(448.0)


def rms_norm(x, residual, weight, eps: float):
    """(h, y) in float64."""
    h = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    return h, h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def linear(a_codes, a_scales, w_codes, w_scales):
    """(y, the sum of the products' magnitudes) in float64."""
    a = decode(a_codes) * spread(np.asarray(a_scales, np.float64), 1, a_codes.shape[0])
    w = decode(w_codes) * spread(np.asarray(w_scales, np.float64), GROUP, w_codes.shape[0])
    return a @ w.T, np.abs(a) @ np.abs(w).T
