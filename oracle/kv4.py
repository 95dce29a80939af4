"""4-bit K/V cache reference (test infrastructure only).

It shares no code with the CUDA library: the rounding is by comparison with
the format's values in float64, and the byte layout comes from the formulas of
``include/ffpa.h``, one byte index per (token, head dim).

The FFPA docs have no cache; the format is an extension of this library:

* a value is an e2m1 level (0, 0.5, 1, 1.5, 2, 3, 4, 6, signed) times the scale
  of its group of 16 along the head dim;
* a scale byte has five exponent bits (bias 15) and three bits of mantissa;
* scale = amax / 6 rounded to nearest even, amax at most 61440; code = x / scale
  rounded to nearest even, saturating; a NaN counts as zero.
"""
from __future__ import annotations

import numpy as np

TILE = 576
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the finite scales, in the order of their bytes: subnormal steps of 2^-17, then 3-bit mantissas
SCALES = np.array([c * 2.0 ** -17 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 18) for c in range(0xF8)])


def _nearest_even(x, grid):
    """Indices of the entries of the ascending `grid` nearest to x >= 0 (ties: the even index; saturating)."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def quantize(x):
    """x [..., D] -> (codes [..., D] 0..15, scale bytes [..., D / 16])."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    amax = np.minimum(np.abs(g).max(-1), 61440.0)
    sc = _nearest_even(amax / 6.0, SCALES)
    s = SCALES[sc][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        # a level is nearest to |x| / s iff level * s (exact) is nearest to |x|: no quotient is formed
        a = np.abs(g)
        best = np.zeros(g.shape, dtype=np.int64)
        for c in range(1, 8):
            mid = (LEVELS[c - 1] + LEVELS[c]) / 2 * s  # exact
            up = (a > mid) | ((a == mid) & (c % 2 == 0))
            best = np.where((s > 0) & up, c, best)
    code = best | np.where(np.signbit(g), 8, 0)
    return code.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def dequantize(code, sc):
    """The values (float64) of codes [..., D] and scale bytes [..., D / 16]."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(sc < 0xF8, SCALES[np.minimum(sc, 0xF7)], np.where(sc == 0xF8, np.inf, np.nan))
    with np.errstate(invalid="ignore"):
        return (v.reshape(*code.shape[:-1], code.shape[-1] // 16, 16) * s[..., None]).reshape(code.shape)


def _bytes(kv: int, token, D: int):
    """(code byte [.., D], odd nibble [D], scale byte [.., D / 16]) within a strip, for places `token` (0..15) in it."""
    s = np.asarray(token)[..., None]
    d = np.arange(D)
    x, c = d % 64, d // 64
    if kv == 0:
        code = ((s % 8) * 4 + x // 16) * 16 + (s // 8) * 8 + (x % 16) // 2
        scale = 512 + (s % 8) * 8 + (x // 16) * 2 + s // 8
    else:
        code = ((x // 8) * 4 + (s % 8) // 2) * 16 + (s // 8) * 8 + (s % 2) * 4 + (x % 8) // 2
        scale = 512 + (x // 16) * 16 + ((s % 8) // 2) * 4 + (s // 8) * 2 + s % 2
    return code + c * TILE, d % 2, (scale + c * TILE)[..., ::16]


def _strip(cache, kv: int, page: int, h: int, place: int):
    return cache[page, kv, h, place // 16].reshape(-1)


def write(cache, table_row, start: int, k, v) -> None:
    """Writes tokens k, v [N, Hkv, D] as cached tokens start .. start + N - 1 of the sequence with blocks `table_row`
    into cache (uint8 ndarray [pages, 2, Hkv, page_size / 16, D / 64, 576]), in place."""
    page_size = 16 * cache.shape[3]
    for kv, x in ((0, k), (1, v)):
        n, H, D = x.shape
        code, sc = quantize(x)
        for i in range(n):
            pos = start + i
            page, place = int(table_row[pos // page_size]), pos % page_size
            at, odd, at_s = _bytes(kv, place % 16, D)
            for h in range(H):
                row = _strip(cache, kv, page, h, place)  # a view
                lo, hi = code[i, h, 0::2], code[i, h, 1::2]
                row[at[0::2]] = lo | (hi << 4)
                row[at_s] = sc[i, h]


def read(cache, table_row, start: int, n: int):
    """Cached tokens start .. start + n - 1 as (k, v) float64 [n, Hkv, D]."""
    pages, _, H, strips, chunks, _ = cache.shape
    D, page_size = 64 * chunks, 16 * strips
    out = []
    for kv in (0, 1):
        y = np.zeros((n, H, D))
        for i in range(n):
            pos = start + i
            page, place = int(table_row[pos // page_size]), pos % page_size
            at, odd, at_s = _bytes(kv, place % 16, D)
            for h in range(H):
                row = _strip(cache, kv, page, h, place)
                y[i, h] = dequantize((row[at] >> (4 * odd)) & 15, row[at_s])
        out.append(y)
    return out[0], out[1]
