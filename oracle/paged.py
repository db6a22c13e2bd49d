"""A paged key/value cache and the attention over it, in float64.

Position p of lane b is slot p % page_size of page tables[b][p // page_size];
column i of lane b is at position cached[b] + i and sees positions up to its
own (the last ``window`` of them, if window > 0).

8-bit numbers stand for y * 2^e with one e for each token and head: the least
integer in -48..48 with top * 2^e >= max |x| (byte e + 127; 255 for what
cannot be held), y = x / 2^e rounded to nearest, ties to even.
"""

import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}
LEAST, MOST = -48, 48


def e4m3_values():
    """The 256 numbers of the e4m3 type, by their bits."""
    out = np.zeros(256)
    for bits in range(256):
        sign, ex, m = -1.0 if bits & 128 else 1.0, (bits >> 3) & 15, bits & 7
        if ex == 15 and m == 7:
            out[bits] = np.nan
        elif ex == 0:
            out[bits] = sign * m * 2.0 ** -9
        else:
            out[bits] = sign * (8 + m) * 2.0 ** (ex - 10)
    return out


def quantise(x, kind):
    """x [..., dim] -> (y [..., dim], byte [...]): the rounded numbers and the exponents'
    bytes; y is NaN where the byte is 255."""
    x = np.asarray(x, np.float64)
    big = np.max(np.abs(x), axis=-1)
    byte = np.full(big.shape, 255, np.int64)
    held = np.isfinite(big) & (big <= TOP[kind] * 2.0 ** MOST)
    e = np.full(big.shape, LEAST)
    while True:  # raise what does not hold the largest number yet
        low = held & (TOP[kind] * 2.0 ** e.astype(np.float64) < np.where(held, big, 0.0))
        if not low.any():
            break
        e[low] += 1
    byte[held] = e[held] + 127
    z = np.where(held[..., None], x, np.nan) * 2.0 ** -e.astype(np.float64)[..., None]
    if kind == "int8":
        return np.round(z), byte
    grid = e4m3_values()[:127]  # ascending magnitudes
    m = np.abs(np.where(np.isnan(z), 0.0, z))
    hi = np.clip(np.searchsorted(grid, m), 1, 126)
    lo = hi - 1
    up = (grid[hi] - m < m - grid[lo]) | ((grid[hi] - m == m - grid[lo]) & (hi % 2 == 0))
    y = np.where(up, grid[hi], grid[lo])
    y = np.where(m == 0, 0.0, y)
    return np.where(np.isnan(z), np.nan, np.copysign(y, z)), byte


def values(y, byte):
    """What stored numbers stand for."""
    byte = np.asarray(byte, np.float64)
    return np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))[..., None] * np.asarray(y, np.float64)


def lane_slots(table, page_size, first, count):
    """(page, slot) of positions first .. first + count - 1 of a lane."""
    p = np.arange(first, first + count)
    return np.asarray(table)[p // page_size], p % page_size


def attention(q, k, v, before, scale, window=0):
    """One lane: q [n, q_heads, dim]; k, v [before + n, kv_heads, dim] by position.

    Returns (out [n, q_heads, dim], lse [n, q_heads], mag, peak): mag is the same sum with
    |v| for v, peak [n, q_heads] the largest sum_d |scale q_d k_d| of a position that is seen."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    per = hq // k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, peak = np.zeros((n, hq)), np.zeros((n, hq))
    for i in range(n):
        end = before + i + 1
        start = max(0, end - window) if window else 0
        for h in range(hq):
            kk, vv = k[start:end, h // per], v[start:end, h // per]
            s = scale * (kk @ q[i, h])
            top = s.max()
            w = np.exp(s - top)
            total = w.sum()
            out[i, h], mag[i, h] = w @ vv / total, w @ np.abs(vv) / total
            lse[i, h] = top + np.log(total)
            peak[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, mag, peak
