"""The 8-bit cache format in float64, from its definition (see include/cb.h, "8-bit paged
cache"). TEST INFRASTRUCTURE ONLY, as the rest of this package.

A row x is y * 2^e: e the least exponent >= -126 with max |x| <= 448 * 2^e over the finite
elements (0 where they are all zero), y = x / 2^e rounded to the nearest e4m3 value, ties to
even; infinities become 448, NaN stays NaN.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """The non-negative finite e4m3 values in ascending order, from the format: 4 exponent bits
    with bias 7, 3 fraction bits, the largest code a NaN."""
    out = [m / 8.0 * 2.0 ** -6 for m in range(8)]
    for e in range(1, 16):
        out += [(1.0 + m / 8.0) * 2.0 ** (e - 7) for m in range(8)]
    return np.array(out[:-1])


_GRID = e4m3_values()


def round_e4m3(x):
    """Nearest e4m3 value of each element, ties to the even code, by search in the grid."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    hi = np.clip(np.searchsorted(_GRID, a, side="left"), 0, len(_GRID) - 1)
    lo = np.clip(hi - 1, 0, None)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(a >= _GRID[-1], len(_GRID) - 1, pick)
    return np.where(np.isnan(x), np.nan, np.copysign(_GRID[pick], x))


def quantise_rows(x):
    """Rows [..., D] -> (y [..., D], e [...]) with the row standing for y * 2^e."""
    x = np.asarray(x, np.float64)
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -126, np.int64)
    while True:  # raise until it fits
        low = top > E4M3_MAX * np.exp2(e.astype(np.float64))
        if not low.any():
            break
        need = np.floor(np.log2(np.where(low, top, 1.0) / E4M3_MAX)).astype(np.int64)
        e = np.where(low, np.maximum(e + 1, need), e)
    e = np.where(top == 0, 0, e)
    return round_e4m3(x / np.exp2(e.astype(np.float64))[..., None]), e


def codes(y, e):
    """The bytes of (y, e): e4m3 codes and scale bytes."""
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    c = np.searchsorted(_GRID, a).astype(np.uint8)
    c = np.where(np.isnan(y), 0x7F, c | (np.signbit(y).astype(np.uint8) << 7)).astype(np.uint8)
    return c, (e + 127).astype(np.uint8)


def values(code, scale):
    """Bytes back to float64 rows."""
    code = np.asarray(code, np.uint8)
    grid = np.concatenate([_GRID, [np.nan]])
    y = np.copysign(grid[code & 0x7F], np.where(code & 0x80, -1.0, 1.0))
    return y * np.exp2(np.asarray(scale, np.float64) - 127.0)[..., None]


def write_kv(code, scale, rows, slot_mapping):
    """Quantise row t into flat slot slot_mapping[t] of (code, scale), in place."""
    nb, bs, hkv, d = code.shape
    c, s = codes(*quantise_rows(rows))
    flat, fs = code.reshape(nb * bs, hkv, d), scale.reshape(nb * bs, hkv)
    for t, slot in enumerate(np.asarray(slot_mapping).tolist()):
        if slot >= 0:
            flat[slot], fs[slot] = c[t], s[t]
