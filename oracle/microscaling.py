"""Microscaled 4-bit operands (OCP MX v1.0: E2M1 values, E8M0 scales, blocks of
32) and the global-norm clip in float64 numpy: test infrastructure, sharing no
code with the HIP path.

Readings (the specification leaves the conversion's scale to the implementer):
  M1  a block's scale is 2^k, k the smallest integer >= -127 with
      max|x| <= 6 * 2^k (nothing saturates; the rule of the 8-bit payload)
  M2  nearest rounding takes ties to the even code; stochastic rounding with a
      byte r goes up (in magnitude) where 256 * fraction > r + 1/2
  M3  a block with an infinity or a NaN has scale byte 255 and zero codes
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def block_exponent(amax: float) -> int:
    """Smallest k >= -127 with amax <= 6 * 2^k."""
    if amax == 0.0:
        return -127
    f, e = math.frexp(amax / 6.0)  # exact enough: verified below against both neighbours
    k = e if f > 0.5 else e - 1
    while amax > math.ldexp(6.0, k):
        k += 1
    while amax <= math.ldexp(6.0, k - 1):
        k -= 1
    return max(k, -127)


def quantize(x: np.ndarray, rand: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray]:
    """(codes, scale bytes) of a rows x cols matrix, blocks along the rows:
    codes rows x (32 * blocks) of 0..15, scale bytes rows x blocks."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    codes = np.zeros((rows, nb * BLOCK), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for i in range(rows):
        for b in range(nb):
            v = x[i, b * BLOCK:(b + 1) * BLOCK]
            if not np.all(np.isfinite(v)):
                scales[i, b] = 255
                continue
            k = block_exponent(float(np.max(np.abs(v))))
            scales[i, b] = k + 127
            a = np.abs(v) * math.ldexp(1.0, -k)
            lo = np.searchsorted(GRID, a, side="right") - 1
            hi = np.minimum(lo + 1, 7)
            gap = np.where(hi > lo, GRID[hi] - GRID[lo], 1.0)
            frac = (a - GRID[lo]) / gap
            if rand is None:
                up = (frac > 0.5) | ((frac == 0.5) & (hi % 2 == 0))
            else:
                up = frac * 256.0 > rand[i, b * BLOCK:(b + 1) * BLOCK].astype(np.float64) + 0.5
            c = np.where(up, hi, lo).astype(np.uint8)
            codes[i, b * BLOCK:b * BLOCK + v.size] = c | (np.signbit(v).astype(np.uint8) << 3)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """float64 values of (codes, scale bytes); a scale byte of 255 is NaN."""
    mag = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return (mag * np.repeat(unit, BLOCK, axis=1))[:, :cols]


def round_values(x: np.ndarray, rand: Optional[np.ndarray] = None) -> np.ndarray:
    x = np.asarray(x)
    return values(*quantize(x, rand), x.shape[1])


def pack_codes(codes: np.ndarray) -> np.ndarray:
    """Two codes to a byte, the even one in the low nibble."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def scale_index(i: int, b: int, cols: int) -> int:
    """Byte of row i, block b among an operand's scale tiles."""
    chunks = -(-cols // 256)
    return ((i // 32) * chunks + b // 8) * 256 + b % 8 // 2 * 64 + i % 16 * 4 + i % 32 // 16 * 2 + b % 2


def pack_scales(scales: np.ndarray, cols: int) -> Tuple[np.ndarray, np.ndarray]:
    """(bytes, which of them are defined): the tiles, where rows past the last
    are left undefined and blocks past the last are zero."""
    rows, nb = scales.shape
    chunks = -(-cols // 256)
    n = -(-rows // 32) * chunks * 256
    out, known = np.zeros(n, np.uint8), np.zeros(n, bool)
    for i in range(rows):
        for b in range(chunks * 8):
            j = scale_index(i, b, cols)
            known[j] = True
            if b < nb:
                out[j] = scales[i, b]
    return out, known


def clip(grads, max_norm: float, scale: float = 1.0):
    """(norm, coefficient, per-tensor norms, outputs) in float64."""
    with np.errstate(invalid="ignore", over="ignore"):
        sq = [float(np.sum((np.asarray(g, np.float64) * scale) ** 2)) for g in grads]
        norm = math.sqrt(sum(sq)) if not any(math.isnan(s) for s in sq) else math.nan
        c = max_norm / (norm + 1e-6)
        coef = math.nan if math.isnan(norm) else (c if c < 1.0 else 1.0)  # 1 for inf / inf: nothing is clipped
        outs = [np.asarray(g, np.float64) * scale * coef for g in grads]
    return norm, coef, [math.sqrt(s) for s in sq], outs
