"""MX FP4 in float64, from the format's definition (OCP Microscaling Formats:
E2M1 elements, blocks of 32 under E8M0 scales)."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

BLOCK = 32
#: magnitudes of the codes 0..7
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def blocks(K: int) -> int:
    return -(-K // BLOCK)


def floor_log2(v: float) -> int:
    """floor(log2 v) of a positive finite float, exactly."""
    m, e = np.frexp(np.float64(v))       # v = m 2^e, m in [0.5, 1)
    return int(e) - 1


def round_code(u: Fraction) -> int:
    """The code nearest to u >= 0, ties to the even code, beyond 6 to 6."""
    grid = [Fraction(g) for g in GRID]
    best = min(abs(u - g) for g in grid)
    near = [i for i, g in enumerate(grid) if abs(u - g) == best]
    return near[0] if len(near) == 1 else next(i for i in near if i % 2 == 0)


# The rounding borders, half way between neighbours; the border itself goes
# to the even code.
_MID = np.array([(a + b) / 2 for a, b in zip(GRID, GRID[1:])])


def _codes(u: np.ndarray) -> np.ndarray:
    a = np.abs(u)
    c = np.zeros(a.shape, np.int64)
    for i, mid in enumerate(_MID):       # between codes i and i + 1
        c += (a >= mid) if (i + 1) % 2 == 0 else (a > mid)
    return c + 8 * np.signbit(u)


def quantize_rows(x: np.ndarray):
    """float rows [M, K] -> (codes uint8 [M, 16 B], scales uint8 [M, B])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    B = blocks(K)
    pad = np.zeros((M, B * BLOCK))
    pad[:, :K] = x
    v = pad.reshape(M, B, BLOCK)
    codes = np.zeros((M, B, BLOCK), np.int64)
    scales = np.zeros((M, B), np.int64)
    top = np.abs(v).max(axis=2, initial=0.0)
    bad = ~np.isfinite(v).all(axis=2)
    for m in range(M):
        for b in range(B):
            if bad[m, b]:
                scales[m, b] = 255
                continue
            e = max(floor_log2(top[m, b]) - 2, -127) if top[m, b] > 0 else -127
            scales[m, b] = e + 127
            codes[m, b] = _codes(np.ldexp(v[m, b], -e))
    flat = codes.reshape(M, B * BLOCK)
    return (flat[:, 0::2] | (flat[:, 1::2] << 4)).astype(np.uint8), scales.astype(np.uint8)


def dequantize_rows(codes: np.ndarray, scales: np.ndarray, K: int | None = None) -> np.ndarray:
    """codes [M, 16 B], scales [M, B] -> float64 [M, K]."""
    M, B = scales.shape
    c = np.stack((codes & 15, codes >> 4), axis=2).reshape(M, B, BLOCK).astype(np.int64)
    s = scales.astype(np.int64)[:, :, None]
    mag = np.array(GRID)[c & 7]
    v = np.ldexp(np.where(c & 8, -mag, mag), np.broadcast_to(s - 127, c.shape))
    v = np.where(s == 255, np.nan, v).reshape(M, B * BLOCK)
    return v if K is None else v[:, :K]


def linear_w4a4(xq, sx, wq, sw):
    """y [M, N] and the condition scale sum |x||w|, float64."""
    x, w = dequantize_rows(xq, sx), dequantize_rows(wq, sw)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def linear_w4a16(x: np.ndarray, wq, sw):
    x = np.asarray(x, np.float64)
    w = dequantize_rows(wq, sw, x.shape[1])
    return x @ w.T, np.abs(x) @ np.abs(w).T


def qk_norm_rope(x, gain, cos, sin, eps, halves: bool):
    """Heads x [T, H, D] float64, gain [D] or None, cos and sin [T, R/2] ->
    (y, the magnitude of the terms each result is the sum of)."""
    x = np.asarray(x, np.float64)
    D, R = x.shape[2], 2 * cos.shape[1]
    y = x / np.sqrt((x * x).sum(axis=2, keepdims=True) / D + eps)
    if gain is not None:
        y = y * np.asarray(gain, np.float64)
    out, mag = y.copy(), np.abs(y)
    for i in range(R // 2):
        p, q = (i, i + R // 2) if halves else (2 * i, 2 * i + 1)
        c, s = cos[:, i, None], sin[:, i, None]
        out[:, :, p] = y[:, :, p] * c - y[:, :, q] * s
        out[:, :, q] = y[:, :, q] * c + y[:, :, p] * s
        mag[:, :, p] = np.abs(y[:, :, p] * c) + np.abs(y[:, :, q] * s)
        mag[:, :, q] = np.abs(y[:, :, q] * c) + np.abs(y[:, :, p] * s)
    return out, mag
