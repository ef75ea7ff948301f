"""GPU: chunk_attention against the 64-bit oracle (kv_util.tolerance)."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import BATCHES, Batch, tolerance
from test_gpu_kv_cache import device_cache, on_gpu

pytestmark = pytest.mark.gpu

# head_dim, KV heads, query heads per KV head, page tokens
SHAPES = [(128, 2, 1, 8), (128, 1, 5, 128), (128, 3, 16, 16), (256, 2, 12, 64), (256, 1, 4, 256), (256, 1, 1, 32)]


def attend(b, caches, window=0, scale=None, table=None, **kw):
    cache = device_cache(b, caches, table)
    q, _, _, ss, ps = on_gpu(b)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    qsa.chunk_attention(q, ss, ps, cache, window=window, scale=scale, out=out, **kw)
    return out


def check(b, got, caches, window=0, scale=None, vmax=6.0):
    want, mag = b.attention(caches, window, scale)
    n = int(b.seq_start[-1])
    got = got.cpu().numpy().astype(np.float64)
    assert np.all(got[n:] == 7.0)                          # rows of no request
    tol = tolerance(want[:n], mag[:n], b.lens, vmax)
    off = np.abs(got[:n] - want[:n])
    assert np.all(off <= tol), (np.argwhere(~(off <= tol))[:4], np.nanmax(off / tol))


def ok():
    st = qsa.get_device_status()
    assert st == qsa.QSA_OK, qsa.status_string(st)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("D,hkv,group,page", SHAPES)
@pytest.mark.parametrize("lens", BATCHES.values(), ids=BATCHES)
def test_matches_the_oracle(lens, D, hkv, group, page, quantised):
    b = Batch(31, lens, hkv=hkv, group=group, head_dim=D, page=page, quantised=quantised)
    caches = b.stored()
    got = attend(b, caches)
    ok()
    check(b, got, caches)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("window", [1, 7, 128, 129, 250, 100000])
@pytest.mark.parametrize("D,hkv,group,page", [(128, 2, 3, 8), (256, 1, 12, 64)])
def test_window(D, hkv, group, page, window, quantised):
    lens = [(1, 513), (90, 127), (129, 400), (1, 3)]
    b = Batch(32, lens, hkv=hkv, group=group, head_dim=D, page=page, quantised=quantised)
    caches = b.stored()
    # what lies before every row's window may be gone: its table entries are
    # dropped (bad pages would be flagged), its slots hold NaN
    k, v, ks, vs = (None if a is None else a.copy() for a in caches)
    table = b.table.copy()
    for r, (n, c) in enumerate(lens):
        lo = max(0, c - n - window + 1)
        table[r, :lo // page] = -1
        for t in range(lo // page * page, lo):
            k[b.table[r, t // page], t % page] = 0x7F if quantised else np.nan
            v[b.table[r, t // page], t % page] = 0x7F if quantised else np.nan
    got = attend(b, (k, v, ks, vs), window, table=table)
    ok()
    check(b, got, caches, window)


@pytest.mark.parametrize("quantised", [False, True])
def test_large_scores(quantised):
    """Scores of tens: one weight near one, the maximum rising along the row."""
    b = Batch(33, [(40, 1000), (1, 900)], hkv=1, group=4, head_dim=256, page=16, quantised=quantised)
    k, v, ks, vs = b.stored()
    if not quantised:
        for t in range(0, 960, 100):                       # ever larger keys along the first request
            k[b.table[0, t // 16], t % 16] *= np.float16(1 + t / 200)
    got = attend(b, (k, v, ks, vs), scale=0.5)
    ok()
    want, mag = b.attention((k, v, ks, vs), 0, 0.5)
    n = int(b.seq_start[-1])
    # scores are scale / head_dim^-0.5 = 8 times those of the derivation, and keys up to
    # 5.8 times as long: 2 * 47 * 2^-12 of sum w |v| in place of 2 * 2^-12
    tol = tolerance(want[:n], mag[:n], b.lens, 6.0) + 94 * 2.0 ** -12 * mag[:n]
    assert np.all(np.abs(got.cpu().numpy()[:n].astype(np.float64) - want[:n]) <= tol)


def test_the_quantised_cache_is_its_fp16_image():
    """Reading back is exact, so attention over the quantised cache equals
    attention over an FP16 cache of the same values."""
    b = Batch(34, [(70, 600), (1, 333)], hkv=2, group=6, head_dim=128, page=32, quantised=True)
    caches = b.stored()
    got = attend(b, caches)
    cache = device_cache(b, caches)
    _, _, _, ss, ps = on_gpu(b)
    image = qsa.KVCache.empty(b.num_pages, b.P, b.hkv, b.D, cache.block_table)
    starts = torch.tensor([0, 600, 933], dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    k, v = qsa.kv_load(starts, zero, 933, cache)
    qsa.kv_store(k, v, starts, zero, image)
    out = torch.full_like(got, 7.0)
    qsa.chunk_attention(on_gpu(b)[0], ss, ps, image, out=out)
    ok()
    assert torch.equal(out, got)


@pytest.mark.parametrize("quantised", [False, True])
def test_bad_page_counts_as_zeros(quantised):
    b = Batch(35, [(20, 300), (2, 50)], hkv=2, group=2, head_dim=256, page=16, quantised=quantised)
    caches = b.stored()
    b.table[0, 3] = b.num_pages                            # the oracle reads zeros there, too
    got = attend(b, caches)
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE
    check(b, got, caches)


def test_bad_requests_are_flagged_and_their_rows_left():
    b = Batch(36, [(6, 40), (5, 5), (4, 30)], hkv=1, group=2, head_dim=128, page=8, quantised=False)
    caches = b.stored()
    for pos in ([-1, 0, 26], [b.max_pages * 8 - 5, 0, 26]):
        cache = device_cache(b, caches)
        q, _, _, ss, _ = on_gpu(b)
        out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
        qsa.chunk_attention(q, ss, torch.tensor(pos, dtype=torch.int32, device="cuda"), cache, out=out)
        assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
        assert torch.all(out[:6] == 7.0)
        want, mag = b.attention(caches)
        off = np.abs(out.cpu().numpy()[6:15].astype(np.float64) - want[6:15])
        assert np.all(off <= tolerance(want[6:15], mag[6:15], b.lens, 6.0))


def test_repeatable_captured_and_on_another_stream():
    b = Batch(37, [(60, 700), (1, 1200)], hkv=2, group=12, head_dim=256, page=64, quantised=False)
    caches = b.stored()
    first = attend(b, caches)
    check(b, first, caches)
    assert torch.equal(first, attend(b, caches))
    q, _, _, ss, ps = on_gpu(b)
    cache = device_cache(b, caches)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = qsa.chunk_attention(q, ss, ps, cache, stream=side)   # output and workspace made here
    side.synchronize()
    n = int(b.seq_start[-1])
    assert torch.equal(got[:n], first[:n])
    ws = qsa.alloc_chunk_attention_workspace(cache, b.T, b.hq)
    ws.random_(0, 256)                                          # nothing in it has to start at zero
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.chunk_attention(q, ss, ps, cache, out=out, ws=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:n], first[:n])
    # the same graph after the batch has moved on: positions are read on the device
    ps.copy_(torch.tensor([600, 1000], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    b.pos_start = np.array([600, 1000], np.int32)
    want, mag = b.attention(caches)
    off = np.abs(out.cpu().numpy()[:n].astype(np.float64) - want[:n])
    assert np.all(off <= tolerance(want[:n], mag[:n], b.lens, 6.0))


def test_a_prompt_in_chunks_through_the_three_calls():
    """A prompt written and attended chunk by chunk, then single tokens: each
    step stores its tokens first; the rows equal those of one whole call."""
    rng = np.random.default_rng(38)
    T, hkv, group, D, P = 333, 2, 6, 128, 16
    x = torch.from_numpy(rng.standard_normal((T, hkv * group + 2 * hkv, D)).astype(np.float16)).cuda()
    table = torch.from_numpy(rng.permutation(40).astype(np.int32)[None, :24]).cuda()
    for quantised in (False, True):
        cache = qsa.KVCache.empty(40, P, hkv, D, table, quantised=quantised)
        outs, at = [], 0
        for n in [100, 1, 128, 101, 1, 1, 1]:
            part = x[at:at + n]
            ss = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            ps = torch.tensor([at], dtype=torch.int32, device="cuda")
            qsa.kv_store(part[:, -2 * hkv:-hkv], part[:, -hkv:], ss, ps, cache)
            outs.append(qsa.chunk_attention(part[:, :-2 * hkv], ss, ps, cache))
            at += n
        assert at == T
        whole = qsa.chunk_attention(x[:, :-2 * hkv], torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                                    torch.zeros(1, dtype=torch.int32, device="cuda"), cache)
        ok()
        parts, whole = torch.cat(outs).double(), whole.double()
        # each is within the rounding of the other: outputs and weights of both sides
        v = qsa.kv_load(torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), T, cache)[1].double()
        assert torch.all((parts - whole).abs() <= 2 * (2.0 ** -11 + 2.0 ** -10 + T * 2.0 ** -25) * v.abs().max())


def test_dense_equals_sparse_when_everything_is_selected():
    """chunk_attention against the framework's sparse-attention consumer with
    every visible position selected."""
    from block_sparse_attention_select_gb300 import workloads as W
    inp = W.make_consumer_inputs("c", seed=22, ctx_tokens=[300, 130], rows_per_req=[6, 3], k=80)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    R = inp.q.shape[0]
    sel = np.full((R, 80), -1, np.int32)
    for r in range(R):
        n = (int(inp.row_token[r]) + 1) // 4
        sel[r, :n] = np.arange(n)
    sparse = qsa.sparse_attention(t(inp.q), t(inp.k_cache), t(inp.v_cache), t(inp.block_table), t(inp.row_req),
                                  t(inp.row_token), t(sel))
    cache = qsa.KVCache(t(inp.k_cache), t(inp.v_cache), t(inp.block_table))
    # each row as a request of its own: one new token at the row's position
    own = qsa.KVCache(cache.k, cache.v, t(inp.block_table[inp.row_req]))
    dense = qsa.chunk_attention(t(inp.q), torch.arange(R + 1, dtype=torch.int32, device="cuda"), t(inp.row_token), own)
    ok()
    mag = np.abs(inp.v_cache.astype(np.float64)).max()
    tol = 2.0 ** -11 * sparse.abs() + (2.0 ** -10 + 300 * 2.0 ** -25) * mag + 2e-4
    assert torch.all((dense.float() - sparse).abs() <= tol)


def reference64(q, k, v, lens, window=0):
    """Attention of contiguous [tokens, heads, dim] requests on the GPU in 64 bits."""
    outs, mags, at, row = [], [], 0, 0
    for n, c in lens:
        kk, vv = k[at:at + c].double(), v[at:at + c].double()
        group = q.shape[1] // k.shape[1]
        kk, vv = (x.repeat_interleave(group, 1).transpose(0, 1) for x in (kk, vv))
        s = torch.matmul(q[row:row + n].double().transpose(0, 1), kk.transpose(1, 2)) * q.shape[2] ** -0.5
        p = torch.arange(c - n, c, device="cuda")[:, None]
        t = torch.arange(c, device="cuda")
        hide = (t > p) | ((t <= p - window) if window else (t > p))
        w = torch.softmax(s.masked_fill(hide, -float("inf")), -1)
        outs.append(torch.matmul(w, vv).transpose(0, 1))
        mags.append(torch.matmul(w, vv.abs()).transpose(0, 1))
        at, row = at + c, row + n
    return torch.cat(outs), torch.cat(mags)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("D,hkv,group,page,lens,window", [
    (128, 8, 4, 128, [(2048, 2048), (1000, 1500)], 0),            # many units of few tiles, ends cut
    (128, 4, 5, 16, [(3001, 3001), (70, 70)], 60),                # one tile or two in every unit
    (256, 2, 12, 64, [(701, 4000), (1, 3500), (300, 300)], 0),
    (256, 4, 3, 8, [(1500, 1500)] * 2, 40),
    (128, 1, 128, 64, [(60, 1000), (1, 1), (2, 129)], 0),         # two query tokens fill a unit
    (256, 8, 1, 256, [(1, 300 + 61 * i) for i in range(50)], 0),  # more requests than a warp
    (128, 2, 7, 32, [(1 + i % 3, 5 + 37 * i) for i in range(70)], 0),
])
def test_many_units(D, hkv, group, page, lens, window, quantised):
    g = torch.Generator(device="cuda").manual_seed(40)
    T, C = sum(n for n, _ in lens), sum(c for _, c in lens)
    need = [-(-c // page) for _, c in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    perm, at = torch.randperm(sum(need), generator=torch.Generator().manual_seed(41)).to(torch.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = qsa.KVCache.empty(sum(need), page, hkv, D, table.cuda(), quantised=quantised)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7F)                               # NaN in both formats
    kv = torch.randn(C, 2 * hkv, D, generator=g, device="cuda", dtype=torch.float16)
    starts = i32(np.concatenate([[0], np.cumsum([c for _, c in lens])]).tolist())
    zero = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    qsa.kv_store(kv[:, :hkv], kv[:, hkv:], starts, zero, cache)
    k, v = qsa.kv_load(starts, zero, C, cache)
    q = torch.randn(T, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
    ss = i32(np.concatenate([[0], np.cumsum([n for n, _ in lens])]).tolist())
    out = qsa.chunk_attention(q, ss, i32([c - n for n, c in lens]), cache, window=window)
    ok()
    want, mag = reference64(q, k, v, lens, window)
    n = max(c for _, c in lens) if not window else window
    tol = 2.0 ** -11 * want.abs() + 2.0 ** -10 * mag + n * 2.0 ** -25 * 6.0 + 2.0 ** -25
    off = (out.double() - want).abs()
    assert torch.all(off <= tol), float((off / tol).max())


def test_binding_refuses():
    b = Batch(39, [(4, 9)], hkv=2, group=2, head_dim=128, page=8, quantised=False)
    cache = device_cache(b, b.stored())
    q, _, _, ss, ps = on_gpu(b)
    with pytest.raises(qsa.QSAError):
        qsa.chunk_attention(q, ss, ps, cache, window=-1)
    with pytest.raises(qsa.QSAError):
        qsa.chunk_attention(q[:, :3], ss, ps, cache)       # three query heads over two KV heads
    with pytest.raises(qsa.QSAError):
        qsa.chunk_attention(q, ss, ps, cache, ws=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        qsa.chunk_attention(q, ss, ps, cache, out=torch.empty(2, 4, 128, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        qsa.chunk_attention(q, ss, ps, cache, out=torch.empty(q.shape, device="cuda"))
    with pytest.raises(ValueError):
        qsa.chunk_attention(q, ss, ps.cpu(), cache)
