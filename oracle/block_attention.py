"""CPU oracle for attention over selected blocks.

TEST INFRASTRUCTURE ONLY, plain numpy in float64, a loop over rows and heads.

Definition: the row at position p attends, for the query heads of KV head g, the
tokens t <= p whose block t // 128 is in sel[row, g] or among the row's `recent`
last blocks (t // 128 > p // 128 - recent), with weights softmax(scale * q . k);
zeros where that is nothing.  Names below 0 or past p // 128 count for nothing.
"""
from __future__ import annotations

import numpy as np

from . import kv_cache

BLOCK = 128


def attended(sel_row, p: int, recent: int) -> np.ndarray:
    """Tokens that a row at position p attends, in order."""
    last = p // BLOCK
    blocks = {int(c) for c in sel_row if 0 <= c <= last} | set(range(max(0, last - recent + 1), last + 1))
    toks = [np.arange(c * BLOCK, min((c + 1) * BLOCK, p + 1)) for c in sorted(blocks)]
    return np.concatenate(toks) if toks else np.zeros(0, int)


def attention(q, sel, seq_start, pos_start, block_table, k, v, k_scale=None, v_scale=None, recent=0, scale=None):
    """q float16 [T, hq, D], sel int [T, hkv, k]; returns (float64 [T, hq, D], and
    the same sum over |values|), NaN in rows of no request."""
    T, hq, D = q.shape
    P, hkv = k.shape[1], k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    group = hq // hkv

    def read(cache, sc, b, toks, g):
        page, slot = block_table[b, toks // P], toks % P
        good = (page >= 0) & (page < cache.shape[0])
        at = np.where(good, page, 0)
        x = cache[at, slot, g].astype(np.float64) if sc is None else kv_cache.dequantise(cache[at, slot, g], sc[at, slot, g])
        return np.where(good[:, None], x, 0.0)

    for b in range(len(pos_start)):
        for r in range(int(seq_start[b]), int(seq_start[b + 1])):
            p = int(pos_start[b]) + r - int(seq_start[b])
            for g in range(hkv):
                toks = attended(sel[r, g], p, recent)
                hs = slice(g * group, (g + 1) * group)
                if len(toks) == 0:
                    out[r, hs] = mag[r, hs] = 0.0
                    continue
                kk, vv = read(k, k_scale, b, toks, g), read(v, v_scale, b, toks, g)
                s = q[r, hs].astype(np.float64) @ kk.T * scale
                e = np.exp(s - s.max(-1, keepdims=True))
                w = e / e.sum(-1, keepdims=True)
                out[r, hs], mag[r, hs] = w @ vv, w @ np.abs(vv)
    return out, mag
