"""GPU: chunk_attention and the K/V cache where they could go wrong: many small
weights, alignment, batches with nothing to do, shared pages, offsets past 32
bits, two calls at once."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import Batch, tolerance
from test_gpu_chunk_attention import attend, check, ok, reference64
from test_gpu_kv_cache import device_cache, on_gpu

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows", [1, 20])                   # few rows, and units of 256
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("D,group", [(128, 4), (256, 2)])
def test_many_small_weights_add_up(D, group, quantised, rows):
    """One large weight at token 0 and 2^18 - 1 weights of 2^-26.2 of it, whose
    values are one: the output is their share of the sum, near 0.0033.  160
    requests over the same pages, so that no request is cut into many parts (a
    part without token 0 has a maximum of its own)."""
    N, P, B, drop = 1 << 18, 128, 160, 26.2
    table = torch.arange(N // P, dtype=torch.int32, device="cuda").flip(0).expand(B, -1).contiguous()
    cache = qsa.KVCache.empty(N // P, P, 1, D, table, quantised=quantised)
    kv = torch.zeros(N, 2, D, dtype=torch.float16, device="cuda")
    kv[0, 0, 0] = 1.0
    kv[1:, 1] = 1.0
    qsa.kv_store(kv[:, :1], kv[:, 1:], i32([0, N]), i32([0]), cache)
    q = torch.zeros(B * rows, group, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    out = qsa.chunk_attention(q, torch.arange(B + 1, dtype=torch.int32, device="cuda") * rows, i32([N - rows] * B), cache,
                              scale=drop * float(np.log(2.0))).double()
    ok()
    n = torch.arange(N - rows, N, device="cuda", dtype=torch.float64).repeat(B)[:, None, None]
    share = n * 2.0 ** -drop
    want = share / (1.0 + share)
    # a weight of 2^-26.2, times 2^7, has FP16 steps of 2^-24: off by at most 2^-32 of the
    # largest weight; the sum, the scores (2^-22 of 26 powers of two) and the output's
    # rounding as ever
    tol = n * 2.0 ** -32 + 2.0 ** -10 * want + 2.0 ** -25
    off = (out - want).abs()
    assert torch.all(off <= tol), (float(off.max()), float(tol.min()))


@pytest.mark.parametrize("quantised", [False, True])
def test_output_aligned_to_16_bytes_only(quantised):
    b = Batch(51, [(150, 400), (1, 77), (33, 33)], hkv=2, group=3, head_dim=128, page=32, quantised=quantised)
    caches = b.stored()
    q, _, _, ss, ps = on_gpu(b)
    flat = torch.full((b.T * b.hq * b.D + 8,), 7.0, dtype=torch.float16, device="cuda")
    out = flat[8:].view(b.T, b.hq, b.D)
    assert out.data_ptr() % 32 == 16
    qsa.chunk_attention(q, ss, ps, device_cache(b, caches), out=out)
    ok()
    check(b, out, caches)
    assert torch.all(flat[:8] == 7.0)
    assert torch.equal(out, attend(b, caches))              # the store's width changes nothing


def test_nothing_to_do():
    """No rows, no requests, only empty requests, a batch that ends before its rows."""
    table = torch.zeros(5, 4, dtype=torch.int32, device="cuda")
    cache = qsa.KVCache.empty(3, 16, 2, 128, table)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    before = cache.k.clone()
    x = torch.randn(6, 4, 128, device="cuda").half()
    for starts, rows in ([0], 6), ([0, 0], 0), ([0] * 6, 6), ([6] * 6, 6), ([0, 0, 0], 0):
        out = torch.full((rows, 4, 128), 7.0, dtype=torch.float16, device="cuda")
        pos = i32([1] * (len(starts) - 1))
        qsa.kv_store(x[:rows, :2], x[:rows, 2:], i32(starts), pos, cache)
        qsa.chunk_attention(x[:rows], i32(starts), pos, cache, out=out)
        qsa.kv_load(i32(starts), pos, rows, cache)
        ok()
        assert torch.all(out == 7.0)
        assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("rows", [1, 3, 30])
def test_the_quantised_cache_of_few_rows_is_its_fp16_image(rows):
    lens = [(rows, 700), (rows, 64), (rows, 333)]
    b = Batch(52, lens, hkv=2, group=5, head_dim=256, page=64, quantised=True)
    caches = b.stored()
    cache = device_cache(b, caches)
    q, _, _, ss, ps = on_gpu(b)
    image = qsa.KVCache.empty(b.num_pages, b.P, b.hkv, b.D, cache.block_table)
    starts, zero = i32([0, 700, 764, 1097]), i32([0, 0, 0])
    qsa.kv_store(*qsa.kv_load(starts, zero, 1097, cache), starts, zero, image)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    qsa.chunk_attention(q, ss, ps, image, out=out)
    ok()
    check(b, out, caches)
    check(b, attend(b, caches), caches)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("tokens", [1, 80])
def test_more_requests_than_threads(tokens, quantised):
    """1,300 requests, one in seven with tokens."""
    lens = [(tokens, tokens + 11 * (i % 13)) if i % 7 == 3 else (0, 0) for i in range(1300)]
    b = Batch(53, lens, hkv=1, group=2, head_dim=128, page=16, quantised=quantised)
    caches = b.stored()
    got = attend(b, caches)
    ok()
    check(b, got, caches)


def test_requests_that_share_a_prefix():
    """Two requests whose tables name the same pages for their first 64 tokens."""
    g = torch.Generator(device="cuda").manual_seed(54)
    hkv, group, D, P = 2, 4, 128, 16
    for quantised in (False, True):
        table = i32([[5, 2, 7, 0, 1, 9], [5, 2, 7, 0, 8, 3]])
        cache = qsa.KVCache.empty(10, P, hkv, D, table, quantised=quantised)
        kv = torch.randn(64 + 30 + 25, 2 * hkv, D, generator=g, device="cuda", dtype=torch.float16)
        qsa.kv_store(kv[:64, :hkv], kv[:64, hkv:], i32([0, 64]), i32([0]), cache)
        qsa.kv_store(kv[64:, :hkv], kv[64:, hkv:], i32([0, 30, 55]), i32([64, 64]), cache)
        q = torch.randn(55, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
        out = qsa.chunk_attention(q, i32([0, 30, 55]), i32([64, 64]), cache).double()
        k, v = qsa.kv_load(i32([0, 94, 183]), i32([0, 0]), 183, cache)
        ok()
        want, mag = reference64(q, k, v, [(30, 94), (25, 89)])
        assert torch.all((out - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -10 * mag + 94 * 2.0 ** -25 * 6.0 + 2.0 ** -25)


@pytest.mark.parametrize("quantised", [False, True])
def test_offsets_past_32_bits(quantised):
    """Pages at the end of a cache of more than 2^32 elements (and, quantised, more
    than 2^32 bytes of codes): stored, read back and attended by both forms."""
    g = torch.Generator(device="cuda").manual_seed(55)
    hkv, group, D, P = 8, 2, 256, 256
    pages = (1 << 32) // (P * hkv * D) + 40
    last = [pages - 1 - 3 * i for i in range(12)]
    cache = qsa.KVCache.empty(pages, P, hkv, D, i32([last[:6], last[6:]]), quantised=quantised)
    lens = [1500, 1411]
    kv = torch.randn(sum(lens), 2 * hkv, D, generator=g, device="cuda", dtype=torch.float16)
    starts, zero = i32([0, lens[0], sum(lens)]), i32([0, 0])
    qsa.kv_store(kv[:, :hkv], kv[:, hkv:], starts, zero, cache)
    k, v = qsa.kv_load(starts, zero, sum(lens), cache)
    ok()
    if quantised:
        off = (k.double() - kv[:, :hkv].double()).abs()
        assert torch.all(off <= torch.maximum(2.0 ** -4 * kv[:, :hkv].double().abs(), torch.full_like(off, 2.0 ** -10 * 2.0 ** -6)))
    else:
        assert torch.equal(k, kv[:, :hkv]) and torch.equal(v, kv[:, hkv:])
    for n in (1, 60):
        q = torch.randn(2 * n, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
        out = qsa.chunk_attention(q, i32([0, n, 2 * n]), i32([c - n for c in lens]), cache).double()
        ok()
        want, mag = reference64(q, k, v, [(n, c) for c in lens])
        assert torch.all((out - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -10 * mag + 1500 * 2.0 ** -25 * 6.0 + 2.0 ** -25)


def test_two_calls_at_once():
    """Two streams, and then two captured graphs, each with its own workspace."""
    made = []
    for seed, lens, quantised in ((56, [(200, 900), (1, 500)], False), (57, [(1, 1200), (1, 800)], True)):
        b = Batch(seed, lens, hkv=2, group=6, head_dim=128, page=32, quantised=quantised)
        caches = b.stored()
        cache = device_cache(b, caches)
        first = attend(b, caches)
        check(b, first, caches)
        made.append((b, cache, on_gpu(b), first, qsa.alloc_chunk_attention_workspace(cache, b.T, b.hq),
                     torch.zeros_like(first), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for b, cache, (q, _, _, ss, ps), _, ws, out, s in made:
            with torch.cuda.stream(s):
                qsa.chunk_attention(q, ss, ps, cache, out=out, ws=ws)
    torch.cuda.synchronize()
    ok()
    graphs = []
    for b, cache, (q, _, _, ss, ps), first, ws, out, s in made:
        n = int(b.seq_start[-1])
        assert torch.equal(out[:n], first[:n])
        out.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qsa.chunk_attention(q, ss, ps, cache, out=out, ws=ws)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, (_, _, _, _, _, _, s) in zip(graphs, made):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    ok()
    for b, _, _, first, _, out, _ in made:
        n = int(b.seq_start[-1])
        assert torch.equal(out[:n], first[:n])


@pytest.mark.parametrize("quantised", [False, True])
def test_requests_out_of_order_are_flagged(quantised):
    """A seq_start that falls: the request that ends before it starts is flagged and
    the others' rows, here without overlap, are right."""
    b = Batch(58, [(10, 90), (4, 4), (20, 50)], hkv=1, group=4, head_dim=128, page=16, quantised=quantised)
    caches = b.stored()
    q, _, _, ss, ps = on_gpu(b)
    cache = device_cache(b, caches)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    qsa.chunk_attention(q, i32([0, 10, 5, 5]), ps, cache, out=out)      # request 1: 10 .. 5, request 2 empty
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    want, mag = b.attention(caches)
    off = np.abs(out.cpu().numpy()[:10].astype(np.float64) - want[:10])
    assert np.all(off <= tolerance(want[:10], mag[:10], b.lens, 6.0))
    assert torch.all(out[10:] == 7.0)


def test_a_window_past_32_bits_is_no_window():
    b = Batch(59, [(70, 300), (1, 40)], hkv=1, group=2, head_dim=128, page=16, quantised=False)
    caches = b.stored()
    first = attend(b, caches)
    for window in (2 ** 31 - 1, 2 ** 32, 2 ** 40 + 5):
        assert torch.equal(attend(b, caches, window=window), first)
    with pytest.raises(qsa.QSAError):
        attend(b, caches, window=-2 ** 32)
    ok()
