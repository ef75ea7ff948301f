"""CPU oracle for the K/V cache operators: writing new tokens into a paged cache
(as FP16 or quantised to E4M3 with a power-of-two scale per token and head),
reading them back, and dense attention of new tokens over the cache.

TEST INFRASTRUCTURE ONLY, plain numpy in float64, loops over tokens and rows.

Definitions: a vector x of one token and head is stored as the nearest E4M3
value (ties to even) of x * 2^-e and the byte e + 127, e the least integer of
[-15, 8] with max |x| <= 448 * 2^e (8 if there is none), codes at most 240 in
magnitude at e = 8.  The row at position p attends tokens max(0, p - window + 1)
.. p (window 0: 0 .. p) with weights softmax(scale * q . k).
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 codes' values (NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = np.nan if (c & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if s else v
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]           # codes 0x00 .. 0x7e, increasing


def encode(y: np.ndarray) -> np.ndarray:
    """Codes of the nearest E4M3 values, ties to the even code, up to +-448."""
    a = np.minimum(np.abs(y), 448.0)
    hi = np.searchsorted(_POSITIVE, a)              # the first value >= a
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, 126)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = np.where(np.isnan(y), 0x7F, code)
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """x float16 [..., D] -> (codes uint8 [..., D], scale bytes uint8 [...])."""
    x = x.astype(np.float64)
    a = np.where(np.isnan(x), 0.0, np.abs(x)).max(-1)
    e = np.full(a.shape, 8)
    for k in range(7, -16, -1):
        e = np.where(a <= 448.0 * 2.0 ** k, k, e)
    y = x * (2.0 ** -e.astype(np.float64))[..., None]
    top = np.where(e == 8, 240.0, 448.0)[..., None]
    y = np.where(np.isnan(y), y, np.clip(y, -top, top))
    return encode(y), (e + 127).astype(np.uint8)


def dequantise(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return _VALUES[codes] * (2.0 ** (scale.astype(np.float64) - 127))[..., None]


def lines(seq_start, pos_start, block_table, page_tokens: int, rows: int):
    """(row, page, slot) of every new token."""
    for b in range(len(pos_start)):
        for r in range(int(seq_start[b]), int(seq_start[b + 1])):
            assert r < rows
            p = int(pos_start[b]) + r - int(seq_start[b])
            yield r, int(block_table[b, p // page_tokens]), p % page_tokens


def store(x, seq_start, pos_start, block_table, cache, scale=None):
    """x float16 [T, hkv, D] into copies of cache (and scale); returns them."""
    cache = cache.copy()
    scale = None if scale is None else scale.copy()
    for r, page, slot in lines(seq_start, pos_start, block_table, cache.shape[1], x.shape[0]):
        if 0 <= page < cache.shape[0]:
            if scale is None:
                cache[page, slot] = x[r]
            else:
                cache[page, slot], scale[page, slot] = quantise(x[r])
    return cache, scale


def load(rows, seq_start, pos_start, block_table, cache, scale=None):
    """float64 [rows, hkv, D] (NaN in rows of no request)."""
    out = np.full((rows,) + cache.shape[2:], np.nan)
    for r, page, slot in lines(seq_start, pos_start, block_table, cache.shape[1], rows):
        if not 0 <= page < cache.shape[0]:
            out[r] = 0.0
        else:
            out[r] = cache[page, slot] if scale is None else dequantise(cache[page, slot], scale[page, slot])
    return out


def attention(q, seq_start, pos_start, block_table, k, v, k_scale=None, v_scale=None, window=0, scale=None):
    """q float16 [T, hq, D]; returns (float64 [T, hq, D], and the same sum over
    |values|: sum_t w_t |v_t|, which bounds what rounding the weights can do)."""
    T, hq, D = q.shape
    P, hkv = k.shape[1], k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b in range(len(pos_start)):
        s0, s1, p0 = int(seq_start[b]), int(seq_start[b + 1]), int(pos_start[b])
        if s1 == s0:
            continue
        end = p0 + s1 - s0
        lo = max(0, p0 - window + 1) if window else 0
        ks, vs = np.zeros((end, hkv, D)), np.zeros((end, hkv, D))
        for t in range(lo, end):
            page, slot = int(block_table[b, t // P]), t % P
            if 0 <= page < k.shape[0]:
                ks[t] = k[page, slot] if k_scale is None else dequantise(k[page, slot], k_scale[page, slot])
                vs[t] = v[page, slot] if v_scale is None else dequantise(v[page, slot], v_scale[page, slot])
        for r in range(s0, s1):
            p = p0 + r - s0
            a = max(0, p - window + 1) if window else 0
            for h in range(hq):
                g = h // (hq // hkv)
                s = ks[a:p + 1, g] @ q[r, h].astype(np.float64) * scale
                e = np.exp(s - s.max())
                w = e / e.sum()
                out[r, h] = w @ vs[a:p + 1, g]
                mag[r, h] = w @ np.abs(vs[a:p + 1, g])
    return out, mag
