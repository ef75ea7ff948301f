"""CPU oracle for a batch's tables from its requests' lengths.

TEST INFRASTRUCTURE ONLY, plain Python, request by request.
"""
from __future__ import annotations

import numpy as np


def tables(new_len, ctx_len, rows, page_tokens, block_table, free_pages, free_count):
    """Returns the arrays of a batch (a dict with the block table among them) and
    whether a request was malformed."""
    P, n = page_tokens, len(new_len)
    table, left = block_table.copy(), int(min(max(free_count, 0), len(free_pages)))
    out = {"seq_start": [0], "pos_start": list(ctx_len), "total_len": []}
    maps = []
    first, bad = n, left != free_count
    for b in range(n):
        new, ctx = int(new_len[b]), int(ctx_len[b])
        if new < 0 or ctx < 0 or new + ctx > table.shape[1] * P:
            bad, new, need = True, 0, 0
        else:
            need = -(-(new + ctx) // P) - -(-ctx // P)
        if first == n and (len(maps) + new > rows or need > left):
            first = b
        if first < n:
            new, need = 0, 0
        for i in range(need):
            left -= 1
            table[b, -(-ctx // P) + i] = free_pages[left]
        maps += [(b, t, (t + 1) // 4, int(table[b, t // P]) * P + t % P) for t in range(ctx, ctx + new)]
        out["seq_start"].append(len(maps))
        out["total_len"].append(ctx + new)
    used = len(maps)
    maps += [(maps[-1][0] if maps else 0, 0, 0, -1)] * (rows - used)
    for i, name in enumerate(("row_req", "row_token", "row_visible", "slot")):
        out[name] = [m[i] for m in maps]
    out["state"], out["block_table"] = [used, left, first], table
    return {k: np.asarray(v, np.int32) for k, v in out.items()}, bad
