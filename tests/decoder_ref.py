"""Float64 references of the decoder layer's operators beside the MoE path (RMS
norm, paged key-value cache, attention of one new token), from their definitions,
on CPU numpy arrays.  They share no code with the library."""
from __future__ import annotations

import numpy as np


def bf16_bits(v) -> np.ndarray:
    """Float values (exact in fp32) -> bf16 bit patterns, round to nearest even; NaN -> 0x7FC0."""
    f = np.asarray(v, np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(f), np.uint16(0x7FC0), r)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_half_step(v) -> np.ndarray:
    """Half the spacing of bf16 values at v: the largest error of a rounding to nearest
    (8 significant bits: 2^-8 of the binade's lower end)."""
    e = np.floor(np.log2(np.maximum(np.abs(np.asarray(v, np.float64)), 2.0 ** -126)))
    return 2.0 ** (e - 8)


_E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if not (c >> 3) & 15 else
                                                (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])
_E4M3[[127, 255]] = np.nan
_POS = _E4M3[:127]  # 0 .. 448, ascending


def e4m3_value(codes) -> np.ndarray:
    return _E4M3[np.asarray(codes, np.uint8)]


def e8m0_value(b) -> np.ndarray:
    b = np.asarray(b, np.uint8)
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))


def e4m3_nearest(v) -> np.ndarray:
    """Code of the E4M3 value nearest to v (|v| <= 448), ties to the even code, by search of the table."""
    a = np.abs(np.asarray(v, np.float64))
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (pick | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def mx8(v) -> tuple[np.ndarray, np.ndarray]:
    """E4M3 codes and E8M0 bytes of groups (the last axis) of float64 values."""
    v = np.asarray(v, np.float64)
    bad = ~np.isfinite(v).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0)).max(-1))
    e = np.full(amax.shape, -127)
    for k in range(-127, 128):  # the smallest exponent that holds the largest value
        e = np.where((amax > 448 * 2.0 ** (k - 1)) & (amax <= 448 * 2.0 ** k), k, e)
    e = np.where(amax > 448 * 2.0 ** 127, 127, e)
    codes = e4m3_nearest(np.where(np.isfinite(v), v, 0) / (2.0 ** e)[..., None])
    return np.where(bad[..., None], 0x7F, codes).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def rmsnorm(x, residual, weight, eps):
    """(a, y) in float64."""
    a = x + (residual if residual is not None else 0.0)
    return a, a / np.sqrt((a * a).mean(-1, keepdims=True) + eps) * weight


def attn(q, k, v, scale):
    """One row: q [D], the seen tokens' k, v [n, D] -> out, lse, and what its error bound needs:
    sum p |v| / l, and the largest of scale * sum |q k|."""
    if len(k) == 0:
        return np.zeros(q.shape[0]), -np.inf, np.zeros(q.shape[0]), 0.0
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = scale * (k @ q)
        m = s.max() if not np.isnan(s).any() else np.nan
        if m == -np.inf:
            return np.zeros(q.shape[0]), -np.inf, np.zeros(q.shape[0]), 0.0
        p = np.exp(s - m)
        l = p.sum()
        return (p @ v) / l, m + np.log(l), (p @ np.abs(v)) / l, float(abs(scale) * (np.abs(k) @ np.abs(q)).max())
