"""fp64 CPU oracle of the paged cache held in 8 bits. Test infrastructure, like ``oracle.attention``.

A row x of d values is d e4m3 numbers y and a code c, a whole number: it stands for y 2^(c - 127). c is 0 for a row of zeros,
255 for one that holds NaN or an infinity, and else floor(log2 max|x|) - 7 + 127, at least 47; y is x 2^(127 - c) rounded to
the nearest e4m3 number, ties to the even one. The numbers are found here by search in a table that is written out from the
format's definition, and attention is ``oracle.paged.attention`` on the rows that the cache stands for.
"""

from __future__ import annotations

import math

import numpy as np


def e4m3_table():
    """The number of each byte: a sign bit, 4 exponent bits biased by 7, 3 fraction bits; no infinities, NaN where all of
    the other bits are set."""
    out = np.empty(256)
    for n in range(256):
        e, f = (n >> 3) & 15, n & 7
        x = f * 2.0**-9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[n] = math.nan if (n & 127) == 127 else (-x if n & 128 else x)
    return out


TABLE = e4m3_table()
_POS = TABLE[:127]  # 0 .. 448, ascending; the index is the byte


def round_e4m3(x):
    """Bytes of the nearest numbers (ties to the even byte) of |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)  # _POS[hi - 1] <= a <= _POS[hi], for a > 0
    lo = hi - 1
    below, above = a - _POS[lo], _POS[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return (np.where(up, hi, lo) + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(x):
    """(bytes [..., d], codes [...]) of rows x."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(x)).max(-1)
    e = np.frexp(np.where(a == 0, 1.0, a))[1] - 1  # floor(log2 a)
    code = np.where(bad, 255, np.where(a == 0, 0, np.maximum(e - 7 + 127, 47)))
    y = round_e4m3(np.where((bad | (a == 0))[..., None], 0.0, x) * 2.0 ** (127.0 - np.where(bad, 127, code))[..., None])
    return y, code.astype(np.uint8)


def values(y, code):
    """The rows that bytes and codes stand for."""
    code = np.asarray(code).astype(np.float64)
    by = np.where(code == 0, 0.0, np.where(code == 255, math.nan, 2.0 ** (code - 127)))
    return TABLE[np.asarray(y)] * by[..., None]


def cache_values(y, codes, which):
    """fp64 [page][slot][head][d] of a cache's keys (0) or values (1); codes are [page][head][slot][2]."""
    return values(y, np.asarray(codes)[..., which].transpose(0, 2, 1))


def places(table, lengths, rows, P, cu=None):
    """(row's index in the tensor of new tokens, page, slot) of each new token that has a place; L counts the tokens."""
    for b, L in enumerate(lengths):
        n = rows if cu is None else int(cu[b + 1] - cu[b])
        for i in range(n):
            j = int(L) - n + i
            if 0 <= j < table.shape[1] * P:
                yield ((b, i) if cu is None else (int(cu[b]) + i,)), int(table[b][j // P]), j % P


def append(k, v, k_cache, v_cache, codes, table, lengths, cu=None):
    """The caches' bytes and codes after the new rows took the last places of their sequences, in place."""
    (ky, kc), (vy, vc) = quantise(k), quantise(v)
    for at, page, slot in places(table, lengths, k.shape[1], k_cache.shape[1], cu):
        k_cache[page, slot], v_cache[page, slot] = ky[at], vy[at]
        codes[page, :, slot, 0], codes[page, :, slot, 1] = kc[at], vc[at]


def read(k, v, k_cache, v_cache, codes, table, lengths, cu=None):
    """Rows k, v filled with the last keys and values of their sequences, in place; others are left."""
    kx, vx = cache_values(k_cache, codes, 0), cache_values(v_cache, codes, 1)
    for at, page, slot in places(table, lengths, k.shape[1], k_cache.shape[1], cu):
        k[at], v[at] = kx[page, slot], vx[page, slot]
