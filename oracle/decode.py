"""float64 oracle of the decode-step operators (test infrastructure only, NumPy, no shared code with
the library): E4M3 and E2M1 values, the RMS norm's output before its 8-bit rounding, weights of a scale
sweep as numbers, the key-value cache's codes, and attention of one token.

Pinned by tests/test_decode_oracle.py.
"""
from __future__ import annotations

import numpy as np

from .lh_oracle import E2M1_GRID, e2m1_index, e4m3_ladder


def e4m3_values(byte) -> np.ndarray:
    """Values of E4M3 bytes (sign, 4 exponent bits, 3 mantissa bits; 0x7F and 0xFF are NaN)."""
    ladder = np.concatenate([[0.0], e4m3_ladder(), [np.nan]])
    b = np.asarray(byte, dtype=np.int64)
    return np.where(b >= 128, -1.0, 1.0) * ladder[b & 127]


def e4m3_codes(x) -> np.ndarray:
    """Bytes of the E4M3 values nearest to x (ties to the even code, saturating), sign kept."""
    x = np.asarray(x, dtype=np.float64)
    values = np.concatenate([[0.0], e4m3_ladder()])
    mids = np.concatenate([(values[1:] + values[:-1]) / 2, [np.inf]])      # exact
    a = np.abs(x)
    idx = np.searchsorted(mids, a, side="left")                            # midpoints below a
    idx = idx + ((idx % 2 == 1) & (a == mids[idx]))                        # a tie above an odd code goes up
    return idx.astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)


def e2m1_values(packed) -> np.ndarray:
    """Values of packed nibbles [..., n/2] -> [..., n], element 2j in the low half of byte j."""
    p = np.asarray(packed, dtype=np.int64)
    n = np.stack([p & 15, p >> 4], axis=-1).reshape(*p.shape[:-1], 2 * p.shape[-1])
    return np.where(n >= 8, -1.0, 1.0) * np.asarray(E2M1_GRID)[n & 7]


def weights(code, fp4, amax, norm: float = 448.0) -> np.ndarray:
    """W [cout, cin] = E2M1 * v * g of one matrix, g = fp32(amax / (6 norm)), unrounded."""
    g = np.float64(np.float32(np.float64(np.float32(amax)) / (6.0 * norm)))
    return e2m1_values(fp4) * np.repeat(e4m3_values(code) * g, 16, axis=-1)


def rms_norm(h, gamma, eps: float, group: int):
    """(y, scale) of rows h [rows, cin]: the normed rows and max|y| / 448 per row or per 128 channels."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(h == 0.0, 0.0, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)) * np.asarray(gamma, dtype=np.float64)
    width = group or h.shape[1]
    scale = np.stack([np.abs(y[:, c:c + width]).max(-1) for c in range(0, h.shape[1], width)], -1) / 448.0
    return y, scale


def cache_unit(amax, four: bool) -> np.ndarray:
    """fp32(amax * fp32(1/2688)) or fp32(amax * fp32(1/448)): the scale of a head."""
    return (np.asarray(amax, dtype=np.float32) * np.float32(1.0 / (2688.0 if four else 448.0))).astype(np.float64)


def cache_codes(x, amax, four: bool):
    """(codes, block scale bytes or None) of x [tokens, heads, dim] with amax [heads]."""
    x = np.asarray(x, dtype=np.float64)
    unit = cache_unit(amax, four)[:, None]
    if not four:
        with np.errstate(divide="ignore", invalid="ignore"):
            return e4m3_codes(np.where(unit > 0, x / unit, np.copysign(0.0, x))), None
    b = x.reshape(*x.shape[:2], x.shape[2] // 16, 16)
    with np.errstate(divide="ignore", invalid="ignore"):
        v = e4m3_values(e4m3_codes(np.where(unit > 0, np.abs(b).max(-1) / (6.0 * unit), 0.0)))
        s = (v * unit).astype(np.float32).astype(np.float64)[..., None]
        idx = np.where(s > 0, e2m1_index(np.where(s > 0, np.abs(b) / s, 0.0)), 0)
    nib = (idx | (np.signbit(b).astype(np.int64) << 3)).reshape(*x.shape[:2], x.shape[2] // 2, 2)
    return (nib[..., 0] | (nib[..., 1] << 4)).astype(np.uint8), e4m3_codes(v)


def cache_values(codes, scales, amax, four: bool) -> np.ndarray:
    """fp32 values (as float64) of codes [..., heads, dim or dim/2] with amax [heads]."""
    unit = cache_unit(amax, four)[:, None]
    if not four:
        return (e4m3_values(codes) * unit).astype(np.float32).astype(np.float64)
    s = (e4m3_values(scales) * unit).astype(np.float32).astype(np.float64)
    return (e2m1_values(codes) * np.repeat(s, 16, axis=-1)).astype(np.float32).astype(np.float64)


def attention(q, k, v, scale: float):
    """(o, sum_t p|v|, max_t sum_i |q_i k_ti|) of one head: q [dim], k, v [tokens, dim]; no tokens give zeros."""
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q), 0.0
    s = k @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max())
