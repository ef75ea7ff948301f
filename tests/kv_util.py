"""Seeded batches for the K/V cache tests: paged caches whose unused slots hold
NaN and whose unused table entries are -1, new tokens as slices of a fused row
array, rows behind the last request."""
from __future__ import annotations

import numpy as np

from oracle import kv_cache as O

# (new tokens, tokens in all) of each request
BATCHES = {
    "one_token": [(1, 1)],
    "two_tokens": [(1, 2), (2, 2)],
    "step": [(1, 129), (1, 1), (1, 700), (1, 128), (1, 64)],
    "chunk": [(37, 300)],
    "prompt": [(261, 261)],
    "mixed": [(1, 513), (0, 40), (90, 127), (0, 0), (3, 3), (129, 400)],
    "tile_ends": [(5, 128), (5, 129), (5, 256), (128, 128), (127, 255)],
}


class Batch:
    def __init__(self, seed, lens, *, hkv, group, head_dim, page, quantised, pad_rows=3):
        rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.hq, self.D, self.P = lens, hkv, hkv * group, head_dim, page
        self.quantised = quantised
        n = np.array([a for a, _ in lens])
        self.seq_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.pos_start = np.array([c - a for a, c in lens], np.int32)
        self.T = int(self.seq_start[-1]) + pad_rows
        need = [-(-c // page) for _, c in lens]
        self.max_pages = max(1, max(need)) + 1
        self.num_pages = sum(need) + 2
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        # one row: hq query vectors, hkv keys, hkv values
        self.fused = rng.standard_normal((self.T, self.hq + 2 * hkv, head_dim)).astype(np.float16)
        self.q = self.fused[:, :self.hq]
        self.k_new, self.v_new = self.fused[:, self.hq:self.hq + hkv], self.fused[:, self.hq + hkv:]
        # the caches before the call: the requests' earlier tokens, NaN elsewhere
        shape = (self.num_pages, page, hkv, head_dim)
        self.ks = self.vs = None
        if quantised:
            self.k, self.v = np.full(shape, 0x7F, np.uint8), np.full(shape, 0x7F, np.uint8)
            self.ks, self.vs = np.full(shape[:3], 200, np.uint8), np.full(shape[:3], 200, np.uint8)
        else:
            self.k, self.v = np.full(shape, np.nan, np.float16), np.full(shape, np.nan, np.float16)
        for b in range(len(lens)):
            for t in range(int(self.pos_start[b])):
                for name, scale in (("k", self.ks), ("v", self.vs)):
                    # token vectors of very unequal size, as caches hold them
                    x = (rng.standard_normal((hkv, head_dim)) * (0.25 if t % 5 else 1.5)).astype(np.float16)
                    at = (self.table[b, t // page], t % page)
                    if quantised:
                        getattr(self, name)[at], scale[at] = O.quantise(x)
                    else:
                        getattr(self, name)[at] = x

    def stored(self):
        """(k, v, k_scale, v_scale) after kv_store of the new tokens."""
        args = (self.seq_start, self.pos_start, self.table)
        k, ks = O.store(self.k_new, *args, self.k, self.ks)
        v, vs = O.store(self.v_new, *args, self.v, self.vs)
        return k, v, ks, vs

    def attention(self, caches, window=0, scale=None):
        k, v, ks, vs = caches
        return O.attention(self.q, self.seq_start, self.pos_start, self.table, k, v, ks, vs, window, scale)


def tolerance(want, mag, lens, vmax):
    """|kernel - 64-bit result| for FP16 outputs: the result's rounding (2^-11 of
    it); the weights' rounding to FP16 for the matrix product (2^-11 of sum w |v|,
    and 2^-25 of |v| for each weight below FP16's normal range); scores summed in
    FP32 over head_dim products (|error| <= head_dim * 2^-24 * scale * sum |q k|,
    below 2^-12 for vectors of unit variance), which moves each weight by that
    much of itself, twice with the normalisation; half of FP16's finest step."""
    n = max(c for _, c in lens)
    return 2.0 ** -11 * np.abs(want) + 2.0 ** -10 * mag + n * 2.0 ** -25 * vmax + 2.0 ** -25
