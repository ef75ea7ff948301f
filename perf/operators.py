"""Cases of the KV-cache operators: kv_store (new tokens into a paged cache, as
FP16 or quantised to E4M3), kv_load (a span of tokens read back as FP16) and
chunk_attention (new tokens attending the paged cache).

A case: op; kv ("fp16" or "e4m3"); reqs requests with up to `new` new tokens
each, up to `ctx` tokens in the cache when they are in; ragged = 0: every
request has exactly these, otherwise the seed of unequal ones; hkv KV heads,
group query heads for each, head_dim, page tokens; window (0: none).
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


def _case(name, op, kv, reqs, new, ctx, ragged, hkv, head_dim, page, group=1, window=0):
    return dict(name=name, op=op, kv=kv, reqs=reqs, new=new, ctx=ctx, ragged=ragged, hkv=hkv, head_dim=head_dim,
                page=page, group=group, window=window)


def listed():
    return [
        # one decode step of a 64-request batch: 64 tokens written, a launch's latency
        _case("store_step_e4m3", "store", "e4m3", 64, 1, 512, 3, 2, 256, 64),
        # the 1,616-row prefill chunk written quantised
        _case("store_chunk_e4m3", "store", "e4m3", 1, 1616, 4096, 0, 2, 256, 64),
        # four prompts of up to 4,096 tokens written as they are, eight KV heads of 128
        _case("store_prompts_fp16", "store", "fp16", 4, 4096, 4096, 5, 8, 128, 128),
        # a whole 184,320-token context read back (a prefix handed to a path that wants FP16)
        _case("load_context_e4m3", "load", "e4m3", 1, 184320, 184320, 0, 2, 256, 64),
        # the last few hundred tokens of 16 requests read back
        _case("load_tails_fp16", "load", "fp16", 16, 300, 2000, 7, 2, 128, 16),
        # a single user's next token over 4,096 tokens: latency, the axis of one row split over the card
        _case("attend_one_fp16", "attend", "fp16", 1, 1, 4096, 0, 2, 256, 64, group=12),
        # a decode step of 64 requests, contexts up to 32,768 tokens: the cache's bytes
        _case("attend_step_fp16", "attend", "fp16", 64, 1, 32768, 11, 2, 256, 64, group=12),
        # the same from the quantised cache
        _case("attend_step_e4m3", "attend", "e4m3", 64, 1, 32768, 12, 2, 256, 64, group=12),
        # the 1,616-row prefill chunk that ends a 29,000-token context: the tensor cores
        _case("attend_chunk_fp16", "attend", "fp16", 1, 1616, 29000, 0, 2, 256, 64, group=12),
        # three requests' chunks, unequal, over quantised contexts
        _case("attend_chunks_e4m3", "attend", "e4m3", 3, 517, 12345, 13, 2, 256, 32, group=12),
        # four whole prompts of 4,096 tokens, 32 query heads over 8 KV heads of 128
        _case("attend_prompts_fp16", "attend", "fp16", 4, 4096, 4096, 0, 8, 128, 128, group=4),
        # a layer with a sliding window of 1,000 tokens, pages of 16, odd lengths
        _case("attend_window_fp16", "attend", "fp16", 2, 1023, 8191, 17, 4, 128, 16, group=5, window=1000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "attend", "attend", "attend"])
    kv = rng.choice(["fp16", "e4m3"])
    head_dim = rng.choice([128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    reqs = _log_int(rng, 1, 64)
    if op != "attend":
        new = _log_int(rng, 1, max(2, 65536 // reqs))
        ctx = new + rng.randrange(0, 2000)
        while reqs * ctx * hkv * head_dim > 184320 * 512:   # no more than the largest listed
            ctx, new = ctx // 2 + 1, max(1, new // 2)
        new = min(new, ctx)
        return _pure(op, kv, reqs, new, ctx, rng.randrange(1 << 20), hkv, head_dim, page)
    new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
    ctx = _log_int(rng, max(16, new), 32768)
    while reqs * new * ctx * hkv * group * head_dim > 1616 * 29000 * 24 * 256 or \
            reqs * ctx * hkv * head_dim > 64 * 32768 * 512:
        if reqs > 1:
            reqs = (reqs + 1) // 2
        else:
            new, ctx = max(1, new // 2), max(16, ctx // 2)
    new = min(new, ctx)
    window = rng.choice([0, 0, 0, _log_int(rng, 1, ctx)])
    return _pure(op, kv, reqs, new, ctx, rng.randrange(1 << 20), hkv, head_dim, page, group, window)


def _pure(*a, **k):
    c = _case("", *a, **k)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and tokens in all of each request."""
    n, c = [case["new"]] * case["reqs"], [case["ctx"]] * case["reqs"]
    if case["ragged"]:
        r = random.Random(case["ragged"])
        n = [r.randint(max(1, case["new"] // 3), case["new"]) for _ in n]
        c = [max(a, r.randint(max(1, case["ctx"] // 16), case["ctx"])) for a in n]
    return n, c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, B, P, H, D = "cuda", case["reqs"], case["page"], case["hkv"], case["head_dim"]
    n, c = _lengths(case)
    T = sum(n)
    starts = [0]
    for a in n:
        starts.append(starts[-1] + a)
    max_pages = -(-max(c) // P)
    used = sum(-(-a // P) for a in c)
    pages = used + 3
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)       # no page past a request's last token
    at = 0
    rows = []
    for b, a in enumerate(c):
        m = -(-a // P)
        rows.append((b, m, at))
        at += m
    table = table.to(dev)
    for b, m, at in rows:
        table[b, :m] = perm[at:at + m]

    def values(rows):
        # keys and values as projections give them: a few channels far larger than the rest
        chan = 1.0 + 5.0 * (torch.rand(D, generator=g, device=dev) < 0.03)
        return (torch.randn(rows, H, D, generator=g, device=dev, dtype=torch.float16) * chan.half())

    quant = case["kv"] == "e4m3"

    def pool():
        x = values(pages * P)                        # stale slots hold what earlier requests left there
        if not quant:
            return x.view(pages, P, H, D), None
        code, scale = _quantise(x)
        return code.view(pages, P, H, D), scale.view(pages, P, H)

    kc, ks = pool()
    vc, vs = pool()
    st = dict(op=case["op"], kc=kc, vc=vc, ks=ks, vs=vs, table=table, T=T, new=max(n), ctx=max(c),
              group=case["group"], window=case["window"], scale=1.0 / math.sqrt(D),
              seq_start=torch.tensor(starts, dtype=torch.int32, device=dev),
              pos_start=torch.tensor([b - a for a, b in zip(n, c)], dtype=torch.int32, device=dev))
    if case["op"] == "store":
        st["k"], st["v"] = values(T), values(T)
    elif case["op"] == "load":
        st["k"] = torch.empty(T, H, D, dtype=torch.float16, device=dev)
        st["v"] = torch.empty_like(st["k"])
    else:
        # queries about as long as keys: scores spread over a few units
        st["q"] = torch.randn(T, H * case["group"], D, generator=g, device=dev, dtype=torch.float16)
        st["out"] = torch.empty_like(st["q"])
    if own:
        from block_sparse_attention_select_gb300 import qsa
        st["cache"] = qsa.KVCache(kc, vc, table, ks, vs)
        if case["op"] == "attend":
            st["ws"] = qsa.alloc_chunk_attention_workspace(st["cache"], T, H * case["group"])
    return st


def _pow2(e):
    """2^e, exact, for the integers -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 codes and scale bytes of the FP16 rows x [..., D]."""
    a = x.abs().amax(-1).float()
    f, e = torch.frexp(a)                            # a = f * 2^e, 0.5 <= f < 1
    e = torch.where(f <= 0.875, e - 9, e - 8)        # the least e with a <= 448 * 2^e
    e = torch.where(a > 0, e, torch.full_like(e, -15)).clamp(-15, 8)
    y = x.float() * _pow2(-e)[..., None]
    top = torch.where(e == 8, 240.0, 448.0)[..., None]
    return torch.minimum(torch.maximum(y, -top), top).to(E4M3), (e + 127).to(torch.uint8)


def _slots(st):
    """Request, page and slot of every new token."""
    row = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["seq_start"][1:], row, right=True)
    pos = (st["pos_start"][b] + row - st["seq_start"][b]).long()
    P = st["kc"].shape[1]
    return b, st["table"][b, pos // P].long(), pos % P


def _bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _value(codes, scale):
    """The 32-bit values of gathered cache rows."""
    return codes.float() if scale is None else codes.float() * _pow2(scale.int() - 127)[..., None]


def _store(st):
    b, page, slot = _slots(st)
    for_k, for_v = (st["k"], None), (st["v"], None)
    if st["ks"] is not None:
        for_k, for_v = _quantise(st["k"]), _quantise(st["v"])
        st["ks"][page, slot] = for_k[1]
        st["vs"][page, slot] = for_v[1]
    _bits(st["kc"])[page, slot] = _bits(for_k[0])
    _bits(st["vc"])[page, slot] = _bits(for_v[0])


def _load(st):
    b, page, slot = _slots(st)

    def read(cache, scale):
        rows = _bits(cache)[page, slot].view(cache.dtype)
        return _value(rows, None if scale is None else scale[page, slot]).half()

    return {"k": read(st["kc"], st["ks"]), "v": read(st["vc"], st["vs"])}


def _attend(st):
    B, P, H, D = st["table"].shape[0], *st["kc"].shape[1:]
    n, L, G = st["new"], st["ctx"], st["group"]
    pos = torch.arange(L, device="cuda")
    page = st["table"][:, pos // P].clamp(min=0).long()

    def read(cache, scale):
        rows = _bits(cache)[page, pos % P].view(cache.dtype)
        return _value(rows, None if scale is None else scale[page, pos % P])          # [B, L, H, D]

    i = torch.arange(n, device="cuda")
    mine = st["pos_start"][:, None] + i                                              # [B, n] positions
    row = (st["seq_start"][:-1, None] + i).clamp(max=st["T"] - 1).long()
    q = st["q"][row].float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    s = torch.matmul(q, read(st["kc"], st["ks"]).permute(0, 2, 3, 1)).mul_(st["scale"])
    hidden = pos > mine[..., None]
    if st["window"]:
        hidden = hidden | (pos <= mine[..., None] - st["window"])
    s.view(B, H, n, G, L).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, read(st["vc"], st["vs"]).permute(0, 2, 1, 3)).div_(total)      # [B, H, n * G, D]
    o = o.view(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H * G, D)
    all_rows = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["seq_start"][1:], all_rows, right=True)
    return o[b, (all_rows - st["seq_start"][b]).long()].half()


def _stored(st):
    """A store's outputs: the caches (and, quantised, the scale bytes) themselves."""
    out = {"k": st["kc"], "v": st["vc"]}
    if st["ks"] is not None:
        out["k_scale"], out["v_scale"] = st["ks"], st["vs"]
    return out


def run(st):
    if own:
        from block_sparse_attention_select_gb300 import qsa
        if st["op"] == "store":
            qsa.kv_store(st["k"], st["v"], st["seq_start"], st["pos_start"], st["cache"])
            return _stored(st)
        if st["op"] == "load":
            k, v = qsa.kv_load(st["seq_start"], st["pos_start"], st["T"], st["cache"], out_k=st["k"], out_v=st["v"])
            return {"k": k, "v": v}
        return qsa.chunk_attention(st["q"], st["seq_start"], st["pos_start"], st["cache"], window=st["window"],
                                   scale=st["scale"], out=st["out"], ws=st["ws"])
    if st["op"] == "store":
        _store(st)
        return _stored(st)
    if st["op"] == "load":
        return _load(st)
    return _attend(st)


def _seen(p, window):
    """Tokens that a row at position p attends."""
    return min(p + 1, window) if window else p + 1


def work(case):
    n, c = _lengths(case)
    H, D, G, W = case["hkv"], case["head_dim"], case["group"], case["window"]
    T = sum(n)
    line = 2 * H * (2 * D if case["kv"] == "fp16" else D + 1)        # cache bytes of one token, K and V
    meta = 4 * (2 * case["reqs"] + 1 + sum(-(-a // case["page"]) for a in c))
    if case["op"] != "attend":
        return {"bytes": T * (line + 2 * H * 2 * D) + meta, "flops": 0}
    # tokens that some row of the request attends; pairs of a row and a token
    span = sum(b - max(0, b - a + 1 - W) if W else b for a, b in zip(n, c))
    pairs = sum(sum(_seen(p, W) for p in range(b - a, b)) for a, b in zip(n, c))
    return {"bytes": span * line + 2 * T * H * G * D * 2 + meta, "flops": 4 * D * H * G * pairs}


# ---- the operators from their definitions, in 64 bits


def _power(e):
    """2^e for whole -200 < e < 200 (library powers are not exact on every device)."""
    return torch.tensor([2.0 ** i for i in range(-200, 200)], dtype=torch.float64, device=e.device)[e.long() + 200]


def _round_e4m3(y):
    """Nearest E4M3 value, ties to even: steps of 2^(floor(log2 |y|) - 3), no finer than 2^-9."""
    _, e = torch.frexp(y)
    step = _power(torch.clamp(e - 1, min=-6) - 3)
    return torch.round(y / step) * step


def _exact_store(st):
    starts, first, table = st["seq_start"].tolist(), st["pos_start"].tolist(), st["table"].tolist()
    P = st["kc"].shape[1]
    out = {}
    for name, cache, x in (("k", st["kc"], st["k"].double()), ("v", st["vc"], st["v"].double())):
        if st["ks"] is not None:
            a = x.abs().amax(-1, keepdim=True)
            best = torch.full_like(a, 8.0)
            for e in range(7, -16, -1):
                best = torch.where(a <= 448.0 * 2.0 ** e, torch.full_like(a, float(e)), best)
            x = _round_e4m3(x * _power(-best))
            x = torch.where(best == 8, x.clamp(-240, 240), x)
        want = cache.double() if cache.dtype == torch.float16 else cache.float().double()
        for b in range(len(first)):
            p = torch.arange(first[b], first[b] + starts[b + 1] - starts[b])
            page = torch.tensor(table[b])[p // P]
            want[page.cuda(), (p % P).cuda()] = x[starts[b]:starts[b + 1]]
        out[name] = want
    if st["ks"] is not None:
        out["k_scale"] = out["v_scale"] = None
    return out


def _span(st, b, lo, hi, cache, scale):
    """Tokens lo .. hi - 1 of request b as 64-bit values [tokens, heads, dim]."""
    P = cache.shape[1]
    whole = st["table"][b, lo // P:(hi - 1) // P + 1].long()
    if cache.dtype == torch.float16:
        x = cache[whole].double()
    else:
        x = cache.view(torch.uint8)[whole].view(E4M3).float().double()
        x = x * _power(scale[whole].long() - 127)[..., None]
    return x.flatten(0, 1)[lo % P:lo % P + hi - lo]


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "store":
        return _exact_store(st)
    starts, first = st["seq_start"].tolist(), st["pos_start"].tolist()
    if st["op"] == "load":
        ends = [first[b] + starts[b + 1] - starts[b] for b in range(len(first))]
        return {name: torch.cat([_span(st, b, first[b], ends[b], cache, scale) for b in range(len(first))])
                for name, cache, scale in (("k", st["kc"], st["ks"]), ("v", st["vc"], st["vs"]))}
    G, W = st["group"], st["window"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(len(first)):
        end = first[b] + starts[b + 1] - starts[b]
        k, v = _span(st, b, 0, end, st["kc"], st["ks"]), _span(st, b, 0, end, st["vc"], st["vs"])
        t = torch.arange(end, device="cuda")
        for r in range(starts[b], starts[b + 1], 256):           # 256 rows of one head at a time
            stop = min(r + 256, starts[b + 1])
            p = torch.arange(first[b] + r - starts[b], first[b] + stop - starts[b], device="cuda")[:, None]
            see = (t <= p) & (t > p - W) if W else t <= p
            for h in range(out.shape[1]):
                s = st["q"][r:stop, h].double() @ k[:, h // G].T * st["scale"]
                s = torch.where(see, s, -math.inf)
                out[r:stop, h] = torch.softmax(s, -1) @ v[:, h // G]
    return out
