"""Cases of the operators that one layer of a block-sparse model runs around the
block scorer: batch_tables (block tables and row maps of a batch from its
requests' lengths), rotary (rotary positions of queries and keys) and
block_attention (new tokens attending the blocks selected for them).

A case: op; reqs requests with up to `new` new tokens each, up to `ctx` tokens
in the cache when they are in; ragged = 0: every request has exactly these,
otherwise the seed of unequal ones; page tokens.  attend: kv ("fp16" or "e4m3"),
hkv KV heads, group query heads for each, head_dim, k selected blocks of 128
tokens, `recent` last blocks, jitter (how much of a selection is the row's own).
rotate: hkv, group, head_dim, rope dims from dim `first` of a head on, the
layout, the scaling and its factor.  tables: rows the batch is padded to, share
of the pages needed that are free (percent).
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
BLOCK = 128
THETA = 10000.0
ORIGINAL = 32768                 # positions before scaling
FAST, SLOW = 32.0, 1.0           # turns of the "parts" scaling's ramp


def _attend_case(name, kv, reqs, new, ctx, ragged, hkv, group, head_dim, page, k, recent=1, jitter=0.5):
    return dict(name=name, op="attend", kv=kv, reqs=reqs, new=new, ctx=ctx, ragged=ragged, hkv=hkv, group=group,
                head_dim=head_dim, page=page, k=k, recent=recent, jitter=jitter)


def _rotate_case(name, reqs, new, ctx, ragged, hkv, group, head_dim, rope, first=0, interleaved=False, scaling="none",
                 factor=1.0):
    return dict(name=name, op="rotate", reqs=reqs, new=new, ctx=ctx, ragged=ragged, hkv=hkv, group=group,
                head_dim=head_dim, rope=rope, first=first, interleaved=interleaved, scaling=scaling, factor=factor)


def _tables_case(name, reqs, new, ctx, ragged, page, rows, free=100):
    return dict(name=name, op="tables", reqs=reqs, new=new, ctx=ctx, ragged=ragged, page=page, rows=rows, free=free)


def listed():
    return [
        # a single user's next token at the end of a 184,320-token context: latency
        _attend_case("attend_one_fp16", "fp16", 1, 1, 184320, 0, 2, 12, 128, 128, 16),
        # a decode step of 64 requests, contexts up to 32,768 tokens: the selected blocks' bytes
        _attend_case("attend_step_fp16", "fp16", 64, 1, 32768, 21, 2, 12, 128, 128, 16),
        # a step of 200 requests from the quantised cache, 256-wide heads, pages of 64
        _attend_case("attend_step_e4m3", "e4m3", 200, 1, 16384, 22, 2, 12, 256, 64, 16),
        # the 1,616-row prefill chunk that ends a 184,320-token context
        _attend_case("attend_chunk_fp16", "fp16", 1, 1616, 184320, 0, 2, 12, 128, 128, 16),
        # three requests' chunks, unequal, over quantised contexts with 256-wide heads
        _attend_case("attend_chunks_e4m3", "e4m3", 3, 517, 12345, 23, 2, 12, 256, 32, 16),
        # four whole prompts of 8,192 tokens, 32 query heads over 4 KV heads
        _attend_case("attend_prompts_fp16", "fp16", 4, 8192, 8192, 0, 4, 8, 128, 128, 16),
        # a decode step of 64 requests, a quarter of each head rotated
        _rotate_case("rotate_step", 64, 1, 32768, 24, 2, 12, 256, 64),
        # the 1,616-row chunk at the end of a context past the original positions
        _rotate_case("rotate_chunk", 1, 1616, 184320, 0, 2, 12, 256, 64, first=192, scaling="parts", factor=8.0),
        # four prompts of 4,096 tokens, whole 128-wide heads, neighbouring dims paired
        _rotate_case("rotate_prompts", 4, 4096, 4096, 0, 8, 4, 128, 128, interleaved=True),
        # a decode step of 64 requests: a launch's latency
        _tables_case("tables_step", 64, 1, 32768, 25, 64, 64),
        # 2,000 requests with drafts of up to 5 tokens, padded, with too few free pages for all
        _tables_case("tables_drafts", 2000, 5, 8192, 26, 16, 8192, free=70),
        # 16 prompts of up to 4,096 tokens that begin their block tables
        _tables_case("tables_prompts", 16, 4096, 4096, 27, 16, 65536),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rotate", "tables"])
    ragged = 1 + rng.randrange(1 << 20)
    if op == "tables":
        reqs = _log_int(rng, 1, 4096)
        new = _log_int(rng, 1, max(2, 65536 // reqs))
        ctx = new + _log_int(rng, 1, 8192)
        rows = min(65536, reqs * new + rng.randrange(0, 600))
        return _pure(_tables_case("", reqs, new, ctx, ragged, rng.choice([8, 16, 32, 64, 128, 256]), rows,
                                  rng.choice([100, 100, 50])))
    group, hkv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), rng.choice([1, 2, 3, 4, 8])
    head_dim = rng.choice([128, 256])
    if op == "rotate":
        reqs = _log_int(rng, 1, 256)
        new = _log_int(rng, 1, max(2, 16384 // reqs))
        ctx = new + _log_int(rng, 1, 100000)
        while reqs * new * hkv * (group + 1) * head_dim > 16384 * 40 * 128:
            new, reqs = max(1, new // 2), max(1, reqs - 1 if new > 1 else reqs // 2)
        head_dim = rng.choice([64, 128, 192, 256]) if new * reqs < 4096 else head_dim
        rope = 16 * rng.randint(1, head_dim // 16)
        scaling = rng.choice(["none", "linear", "base", "parts"])
        return _pure(_rotate_case("", reqs, new, ctx, ragged, hkv, group, head_dim, rope,
                                  first=8 * rng.randint(0, (head_dim - rope) // 8), interleaved=rng.random() < 0.5,
                                  scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.5])))
    kv = rng.choice(["fp16", "e4m3"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    k = _log_int(rng, 1, 64)
    reqs = _log_int(rng, 1, 200)
    new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 8192)
    ctx = _log_int(rng, max(16, new), 65536)
    # no more products, cache or scores of blocks than the largest listed ones
    while reqs * new * min(k * BLOCK, ctx) * hkv * max(group, 4) * head_dim > 32768 * 1024 * 32 * 128 or \
            reqs * ctx * hkv * head_dim > 200 * 16384 * 512 or reqs * new * hkv * (ctx // BLOCK + 1) > 32768 * 4 * 64:
        if reqs > 1:
            reqs = (reqs + 1) // 2
        else:
            new, ctx = max(1, new // 2), max(16, ctx // 2)
    new = min(new, ctx)
    return _pure(_attend_case("", kv, reqs, new, ctx, ragged, hkv, group, head_dim, page, k,
                              recent=rng.choice([0, 1, 1, 2]), jitter=rng.choice([0.25, 0.5, 1.0])))


def _pure(case):
    del case["name"]
    return case


def _lengths(case):
    """New tokens and tokens in all of each request."""
    n, c = [case["new"]] * case["reqs"], [case["ctx"]] * case["reqs"]
    if case["ragged"]:
        r = random.Random(case["ragged"])
        least = 0 if case["op"] == "tables" and case["new"] > 1 else max(1, case["new"] // 3)
        n = [r.randint(least, case["new"]) for _ in n]
        c = [max(a, r.randint(max(1, case["ctx"] // 16), case["ctx"])) for a in n]
    return n, c


def _starts(n):
    out = [0]
    for a in n:
        out.append(out[-1] + a)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"attend": _prepare_attend, "rotate": _prepare_rotate, "tables": _prepare_tables}[case["op"]](case, g)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- inputs


def _prepare_tables(case, g):
    n, c = _lengths(case)
    P, B = case["page"], case["reqs"]
    have = [-(-(b - a) // P) for a, b in zip(n, c)]
    need = [-(-b // P) for b in c]
    fresh = sum(need) - sum(have)
    free = max(1, fresh * case["free"] // 100) if case["free"] < 100 else fresh + 7
    pages = sum(need) + 64
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    max_pages = max(need) + 1
    used = _int32(have)
    first = (torch.cumsum(used, 0) - used).long()
    col = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < used[:, None], perm[at], -1).to(torch.int32)
    # the list's end is where pages are taken from; slots past the count hold old numbers
    st = dict(op="tables", new_len=_int32(n), ctx_len=_int32([b - a for a, b in zip(n, c)]), table=table, page=P,
              rows=case["rows"], free_pages=perm[sum(have):].contiguous(), free_count=_int32([free]))
    if own:
        from block_sparse_attention_select_gb300 import qsa
        st["batch"] = qsa.Batch.empty(B, case["rows"], "cuda")
    return st


def _frequencies(case, device):
    """Angle per position of each pair, in 64 bits, and the amplitude."""
    n, s = case["rope"], case["factor"]
    j = torch.arange(n // 2, dtype=torch.float64, device=device)
    theta = THETA * s ** (n / (n - 2)) if case["scaling"] == "base" else THETA
    f = torch.exp(j * (-2.0 / n * math.log(theta)))
    amplitude = 1.0
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "parts":
        turns = ORIGINAL * f / (2.0 * math.pi)
        keep = ((turns - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / s)
        amplitude = 0.1 * math.log(s) + 1.0
    return f, amplitude


def _prepare_rotate(case, g):
    n, c = _lengths(case)
    H, G, D, T = case["hkv"], case["group"], case["head_dim"], sum(n)
    # queries and keys are slices of a fused projection's rows
    fused = torch.randn(T, H * (G + 2), D, generator=g, device="cuda", dtype=torch.float16)
    q, k = fused[:, :H * G], fused[:, H * G:H * (G + 1)]
    st = dict(op="rotate", q=q, k=k, seq_start=_int32(_starts(n)), pos_start=_int32([b - a for a, b in zip(n, c)]),
              first=case["first"], interleaved=case["interleaved"],
              out_q=torch.empty(T, H * G, D, dtype=torch.float16, device="cuda"),
              out_k=torch.empty(T, H, D, dtype=torch.float16, device="cuda"))
    positions = max(c)
    if own:
        from block_sparse_attention_select_gb300 import qsa
        scaling = None
        if case["scaling"] != "none":
            scaling = qsa.RopeScaling(case["scaling"], case["factor"], original=ORIGINAL, fast=FAST, slow=SLOW,
                                      amplitude=_frequencies(case, "cpu")[1])
        st["table"] = qsa.rotary_table(positions, case["rope"], THETA, scaling)
    else:
        f, amplitude = _frequencies(case, "cuda")
        angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
        st["table"] = torch.cat([angle.cos() * amplitude, angle.sin() * amplitude], 1).float()
    return st


def _selection(case, n, c, g):
    """The blocks that a scorer picks for each row: a request's blocks differ in
    weight, the weights drift along its rows, and each row has its own part."""
    H, k = case["hkv"], case["k"]
    sel = torch.full((sum(n), H, k), -1, dtype=torch.int32, device="cuda")
    at = 0
    for a, b in zip(n, c):
        nb = -(-b // BLOCK)
        x = torch.arange(a, device="cuda") / 32.0
        lo = x.long()
        anchors = torch.randn(a // 32 + 2, H, nb, generator=g, device="cuda")
        score = torch.lerp(anchors[lo], anchors[lo + 1], (x - lo)[:, None, None])
        score += torch.randn(H, nb, generator=g, device="cuda")
        score += case["jitter"] * torch.randn(a, H, nb, generator=g, device="cuda")
        last = (b - a + torch.arange(a, device="cuda")) // BLOCK
        score.masked_fill_((torch.arange(nb, device="cuda") > last[:, None])[:, None, :], -math.inf)
        val, idx = torch.topk(score, min(k, nb), dim=-1)
        sel[at:at + a, :, :min(k, nb)] = torch.where(val == -math.inf, -1, idx).to(torch.int32)
        at += a
    return sel


def _prepare_attend(case, g):
    dev, B, P, H, D = "cuda", case["reqs"], case["page"], case["hkv"], case["head_dim"]
    n, c = _lengths(case)
    T = sum(n)
    need = [-(-a // P) for a in c]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    count = _int32(need)
    col = torch.arange(max(need), device=dev)
    at = ((torch.cumsum(count, 0) - count).long()[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < count[:, None], perm[at], -1).to(torch.int32)

    def values(rows):
        # keys and values as projections give them: a few channels far larger than the rest
        chan = 1.0 + 5.0 * (torch.rand(D, generator=g, device=dev) < 0.03)
        return (torch.randn(rows, H, D, generator=g, device=dev, dtype=torch.float16) * chan.half())

    def pool():
        x = values(pages * P)                        # stale slots hold what earlier requests left there
        if case["kv"] == "fp16":
            return x.view(pages, P, H, D), None
        code, scale = _quantise(x)
        return code.view(pages, P, H, D), scale.view(pages, P, H)

    kc, ks = pool()
    vc, vs = pool()
    st = dict(op="attend", kc=kc, vc=vc, ks=ks, vs=vs, table=table, scale=1.0 / math.sqrt(D), recent=case["recent"],
              seq_start=_int32(_starts(n)), pos_start=_int32([b - a for a, b in zip(n, c)]),
              sel=_selection(case, n, c, g),
              q=torch.randn(T, H * case["group"], D, generator=g, device=dev, dtype=torch.float16))
    st["out"] = torch.empty_like(st["q"])
    if own:
        from block_sparse_attention_select_gb300 import qsa
        st["cache"] = qsa.KVCache(kc, vc, table, ks, vs)
        st["ws"] = qsa.alloc_block_attention_workspace(st["cache"], T, H * case["group"], case["k"], case["recent"])
    return st


def _pow2(e):
    """2^e, exact, for the integers -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 codes and scale bytes of the FP16 rows x [..., D], whose magnitudes are ordinary."""
    _, e = torch.frexp(x.abs().amax(-1).float())
    e = (e - 8).clamp(-15, 8)                        # every value below 256 * 2^e
    return (x.float() * _pow2(-e)[..., None]).to(E4M3), (e + 127).to(torch.uint8)


# ----------------------------------------------------------- plain forms


def _rows(seq_start, rows):
    """Request of every row (the last one's number for rows behind it)."""
    row = torch.arange(rows, device="cuda", dtype=torch.int32)
    return row, torch.searchsorted(seq_start[1:], row, right=True)


def _tables(st):
    new, ctx, P, table, rows = st["new_len"], st["ctx_len"], st["page"], st["table"], st["rows"]
    B = new.shape[0]
    have, need = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    fresh = need - have
    row_end, page_end = torch.cumsum(new, 0), torch.cumsum(fresh, 0)
    served = (row_end <= rows) & (page_end <= st["free_count"])
    n = torch.where(served, new, 0)
    seq_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    seq_start[1:] = torch.cumsum(n, 0)
    col = torch.arange(table.shape[1], device="cuda")
    take = (page_end - fresh)[:, None] + col - have[:, None]
    page = st["free_pages"][(st["free_count"] - 1 - take).clamp(0, st["free_pages"].shape[0] - 1)]
    put = served[:, None] & (col >= have[:, None]) & (col < need[:, None])
    table.copy_(torch.where(put, page, table))
    row, b = _rows(seq_start, rows)
    inside = row < seq_start[-1]
    b = torch.where(inside, b, torch.searchsorted(seq_start[1:], seq_start[-1:] - 1, right=True))   # the last row's
    tok = torch.where(inside, ctx[b] + row - seq_start[b], 0).to(torch.int32)
    slot = torch.where(inside, table[b, (tok // P).long()] * P + tok % P, -1)
    return {"block_table": table, "seq_start": seq_start, "pos_start": ctx.clone(), "total_len": ctx + n,
            "row_req": b.to(torch.int32), "row_token": tok,
            "row_visible": torch.where(inside, (tok + 1) // 4, 0).to(torch.int32), "slot": slot.to(torch.int32),
            "state": torch.stack([seq_start[-1], st["free_count"][0] - torch.where(served, fresh, 0).sum(),
                                  served.sum()]).to(torch.int32)}


def _rotated(x, cos, sin, first, interleaved):
    out = x.float()
    part = out[..., first:first + 2 * cos.shape[-1]]
    if interleaved:
        a, b = part[..., 0::2].clone(), part[..., 1::2].clone()
        part[..., 0::2], part[..., 1::2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = part.chunk(2, -1)
        part.copy_(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))
    return out.half()


def _rotate(st):
    row, b = _rows(st["seq_start"], st["q"].shape[0])
    cos, sin = st["table"][(st["pos_start"][b] + row - st["seq_start"][b]).long()][:, None].chunk(2, -1)
    return {name: _rotated(st[name], cos, sin, st["first"], st["interleaved"]) for name in ("q", "k")}


def _attend(st):
    P, H, D = st["kc"].shape[1:]
    T, hq = st["q"].shape[:2]
    G = hq // H
    row, b = _rows(st["seq_start"], T)
    pos = (st["pos_start"][b] + row - st["seq_start"][b]).long()
    last = (pos // BLOCK)[:, None, None].expand(-1, H, -1)
    blocks = torch.cat([st["sel"].long()] + [last - i for i in range(st["recent"])], -1).sort(-1).values
    twice = torch.zeros_like(blocks, dtype=torch.bool)
    twice[..., 1:] = blocks[..., 1:] == blocks[..., :-1]
    blocks = torch.where(twice, -1, blocks)
    out = torch.empty_like(st["q"])
    step = max(1, (1 << 28) // (blocks.shape[-1] * BLOCK * D))

    def read(cache, scale, page, slot, h):
        x = cache.view(torch.uint8)[page, slot, h].view(E4M3) if scale is not None else cache[page, slot, h]
        return x.float() if scale is None else x.float() * _pow2(scale[page, slot, h].int() - 127)[..., None]

    for r in range(0, T, step):
        s = slice(r, min(r + step, T))
        for h in range(H):
            tok = (blocks[s, h, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)      # [rows, L]
            hidden = (tok < 0) | (tok > pos[s, None])
            tok = torch.where(hidden, 0, tok)
            page, slot = st["table"][b[s, None], tok // P].long(), tok % P
            q = st["q"][s, h * G:(h + 1) * G].float()
            w = torch.matmul(q, read(st["kc"], st["ks"], page, slot, h).transpose(1, 2)).mul_(st["scale"])
            w.masked_fill_(hidden[:, None, :], -math.inf)
            w.sub_(w.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
            total = w.sum(-1, keepdim=True)
            v = read(st["vc"], st["vs"], page, slot, h).masked_fill_(hidden[:, :, None], 0.0)
            o = torch.matmul(w, v) / torch.where(total > 0, total, 1.0)
            out[s, h * G:(h + 1) * G] = o.half()
    return out


def run(st):
    op = st["op"]
    if not own:
        return {"tables": _tables, "rotate": _rotate, "attend": _attend}[op](st)
    from block_sparse_attention_select_gb300 import qsa
    if op == "tables":
        b = qsa.batch_tables(st["new_len"], st["ctx_len"], st["free_pages"], st["free_count"], st["table"], st["page"],
                             st["batch"])
        return {"block_table": st["table"], "seq_start": b.seq_start, "pos_start": b.pos_start,
                "total_len": b.total_len, "row_req": b.row_req, "row_token": b.row_token,
                "row_visible": b.row_visible, "slot": b.slot, "state": b.state}
    if op == "rotate":
        q, k = qsa.rotary(st["q"], st["k"], st["seq_start"], st["pos_start"], st["table"], first=st["first"],
                          interleaved=st["interleaved"], out_q=st["out_q"], out_k=st["out_k"])
        return {"q": q, "k": k}
    return qsa.block_attention(st["q"], st["sel"], st["seq_start"], st["pos_start"], st["cache"], recent=st["recent"],
                               scale=st["scale"], out=st["out"], ws=st["ws"])


def work(case):
    n, c = _lengths(case)
    T, B = sum(n), case["reqs"]
    if case["op"] == "tables":
        fresh = sum(-(-b // case["page"]) - -(-(b - a) // case["page"]) for a, b in zip(n, c))
        return {"bytes": 4 * (5 * B + 1 + 2 * fresh * case["free"] // 100 + 4 * case["rows"] + 4), "flops": 0}
    H, G, D = case["hkv"], case["group"], case["head_dim"]
    if case["op"] == "rotate":
        return {"bytes": 4 * T * H * (G + 1) * D + 4 * T * case["rope"] + 8 * B,
                "flops": 3 * T * H * (G + 1) * case["rope"]}
    # A row attends min(its blocks, all it sees); a request reads at least what one of its rows attends.
    k = case["k"] * BLOCK
    line = 2 * H * (2 * D if case["kv"] == "fp16" else D + 1)        # cache bytes of one token, K and V
    span = sum(min(k, b) for b in c)
    pairs = sum(sum(min(k, p + 1) for p in range(b - a, b)) for a, b in zip(n, c))
    meta = 4 * (2 * B + 1 + T * H * case["k"])
    return {"bytes": span * line + 2 * T * H * G * D * 2 + meta, "flops": 4 * D * H * G * pairs}


# ---- the operators from their definitions, in 64 bits


def exact(case, seed):
    if case["op"] == "attend":
        n, c = _lengths(case)
        if sum(a * b for a, b in zip(n, c)) * case["hkv"] * case["group"] * case["head_dim"] * 4 > 12e12:
            return None                              # too long: every score of every row, in 64 bits
    return {"tables": _exact_tables, "rotate": _exact_rotate, "attend": _exact_attend}[case["op"]](case, prepare(case, seed))


def _exact_tables(case, st):
    new, ctx, P = st["new_len"].tolist(), st["ctx_len"].tolist(), case["page"]
    table, free, left = st["table"].tolist(), st["free_pages"].tolist(), int(st["free_count"])
    out = {"seq_start": [0], "pos_start": ctx, "total_len": [], "row_req": [], "row_token": [], "slot": []}
    rows, served, open_ = 0, 0, True
    for b, (a, p) in enumerate(zip(new, ctx)):
        have, need = -(-p // P), -(-(p + a) // P)
        open_ = open_ and rows + a <= case["rows"] and need - have <= left
        if not open_:
            a = 0
        else:
            served += 1
            for i in range(have, need):
                left -= 1
                table[b][i] = free[left]
        for t in range(p, p + a):
            out["row_req"].append(b)
            out["row_token"].append(t)
            out["slot"].append(table[b][t // P] * P + t % P)
        rows += a
        out["seq_start"].append(rows)
        out["total_len"].append(p + a)
    out["row_visible"] = [(t + 1) // 4 for t in out["row_token"]]
    for name, nothing in (("row_req", out["row_req"][-1] if rows else 0), ("row_token", 0), ("row_visible", 0), ("slot", -1)):
        out[name] += [nothing] * (case["rows"] - rows)
    out["block_table"], out["state"] = table, [rows, left, served]
    return {name: _int32(x) for name, x in out.items()}


def _exact_rotate(case, st):
    n, c = _lengths(case)
    pos = torch.cat([torch.arange(b - a, b, dtype=torch.float64, device="cuda") for a, b in zip(n, c)])
    f, amplitude = _frequencies(case, "cuda")
    turn = torch.polar(torch.full((len(pos), len(f)), amplitude, dtype=torch.float64, device="cuda"), pos[:, None] * f)
    lo, hi = case["first"], case["first"] + case["rope"]
    out = {}
    for name in ("q", "k"):
        y = st[name].double()
        x = y[..., lo:hi].unflatten(-1, (-1, 2)) if case["interleaved"] else y[..., lo:hi].unflatten(-1, (2, -1)).mT
        z = torch.view_as_real(torch.view_as_complex(x.contiguous()) * turn[:, None])
        y[..., lo:hi] = (z if case["interleaved"] else z.mT).flatten(-2)
        out[name] = y
    return out


def _exact_attend(case, st):
    starts, first, sel = st["seq_start"].tolist(), st["pos_start"].tolist(), st["sel"].long()
    P, H, D = st["kc"].shape[1:]
    G, recent = case["group"], case["recent"]
    power = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(len(first)):
        end = first[b] + starts[b + 1] - starts[b]
        pages = st["table"][b, :(end - 1) // P + 1].long()
        t = torch.arange(end, device="cuda")

        def span(cache, scale, h):
            if scale is None:
                return cache[pages, :, h].flatten(0, 1)[:end].double()
            x = cache.view(torch.uint8)[pages, :, h].view(E4M3).float().double() * power[scale[pages, :, h].long()][..., None]
            return x.flatten(0, 1)[:end]

        for h in range(H):
            k, v = span(st["kc"], st["ks"], h), span(st["vc"], st["vs"], h)
            for r in range(starts[b], starts[b + 1], 64):
                stop = min(r + 64, starts[b + 1])
                p = torch.arange(first[b] + r - starts[b], first[b] + stop - starts[b], device="cuda")[:, None]
                member = torch.zeros(stop - r, end // BLOCK + 2, dtype=torch.bool, device="cuda")
                mine = sel[r:stop, h]
                member.scatter_(1, torch.where(mine < 0, end // BLOCK + 1, mine), True)
                see = member[:, t // BLOCK] | (t // BLOCK > p // BLOCK - recent)
                see = see & (t <= p)
                s = torch.einsum("rgd,td->rgt", st["q"][r:stop, h * G:(h + 1) * G].double(), k) * st["scale"]
                w = torch.nan_to_num(torch.softmax(torch.where(see[:, None], s, -math.inf), -1))
                out[r:stop, h * G:(h + 1) * G] = w @ v
    return out
