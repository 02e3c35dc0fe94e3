"""CPU oracle of the 8-bit key / value cache, straight from its definition (numpy float64; shares no code with the
GPU path).  A cache is codes [pages, page size, groups, dim] and scale bytes [pages, groups, blocks], both uint8."""

from __future__ import annotations

import math

import numpy as np

LEAST, MOST, BIAS = -110, 120, 127
LARGEST = 240 * 2.0 ** MOST  # larger finite magnitudes are written as this

# the magnitudes of e4m3 by code: subnormals are multiples of 2^-9, the largest is 448, code 127 is NaN
MAGNITUDES = np.array([m * 2.0 ** -9 if p == 0 else (8 + m) * 2.0 ** (p - 10) for p in range(16) for m in range(8)])
MAGNITUDES[127] = np.nan


def encode(x):
    """Codes of the nearest e4m3 numbers, ties to the even code; anything not finite is NaN (0x7f)."""
    x = np.asarray(x, np.float64)
    size = np.abs(np.where(np.isfinite(x), x, 0.0))
    middle = (MAGNITUDES[1:127] + MAGNITUDES[:126]) / 2
    low, high = np.searchsorted(middle, size, "left"), np.searchsorted(middle, size, "right")
    code = np.where(low % 2 == 0, low, high)
    code = code + np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def decode(codes):
    codes = np.asarray(codes)
    return np.where(codes >= 128, -1.0, 1.0) * MAGNITUDES[codes % 128]


def least_exponent(amax):
    """The least exponent in the scales' range with amax <= 448 * 2^e."""
    e = LEAST
    if amax > 0:
        e = max(LEAST, math.frexp(amax)[1] - 10)
        while amax > 448 * 2.0 ** e:
            e += 1
    return min(e, MOST)


def write(codes, scales, block, x, length, pages):
    """The tokens x [n, groups, dim] of one row to positions length, length + 1, ...; pages[p] holds positions
    p * page size ... (None: no page).  Changes codes and scales in place."""
    x = np.asarray(x, np.float64)
    size, end = codes.shape[1], length + x.shape[0]
    for first in range(length // block * block, end, block):
        page, r = pages[first // size], first % size
        if page is None:
            continue
        a, b = max(first, length), min(first + block, end)
        for g in range(codes.shape[2]):
            new = x[a - length:b - length, g]
            new = np.where(np.isfinite(new), np.clip(new, -LARGEST, LARGEST), new)
            e = least_exponent(np.abs(np.where(np.isfinite(new), new, 0.0)).max())
            if first < length:
                had = int(scales[page, g, r // block]) - BIAS
                if e > had:
                    old = codes[page, r:r + a - first, g]
                    codes[page, r:r + a - first, g] = encode(decode(old) * 2.0 ** (had - e))
                e = max(e, had)
            codes[page, r + a - first:r + b - first, g] = encode(new * 2.0 ** -e)
            scales[page, g, r // block] = e + BIAS


def read(codes, scales, block, begin, end, pages):
    """What positions begin .. end - 1 of a row stand for, [end - begin, groups, dim]; zero where there is no page."""
    out = np.zeros((end - begin, *codes.shape[2:]))
    size = codes.shape[1]
    for j in range(begin, end):
        page = pages[j // size] if 0 <= j < len(pages) * size else None
        if page is not None:
            r = j % size
            out[j - begin] = decode(codes[page, r]) * 2.0 ** (scales[page, :, r // block, None].astype(np.int64) - BIAS)
    return out


def visible(tokens, length, window, sinks):
    """[tokens, length + tokens] truth values: which positions each new token's query sees."""
    i, j = length + np.arange(tokens)[:, None], np.arange(length + tokens)[None]
    return (j <= i) & ((window == 0) | (j > i - window) | (j < sinks))


def step(q, k, v, seen, scale):
    """Queries [tokens, heads, dim] over positions k, v [n, groups, dim] that `seen` [tokens, n] allows: the result
    and the sums of p |v|, both [tokens, heads, dim]; zero rows where nothing is seen."""
    q = np.asarray(q, np.float64)
    share = q.shape[1] // k.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    for t in range(q.shape[0]):
        if not seen[t].any():
            continue
        for h in range(q.shape[1]):
            kk, vv = k[seen[t], h // share], v[seen[t], h // share]
            z = kk @ q[t, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[t, h], size[t, h] = p @ vv, p @ np.abs(vv)
    return out, size
