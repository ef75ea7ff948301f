"""GPU: kv_store and kv_load against the oracle, bit for bit."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import BATCHES, Batch
from oracle import kv_cache as O

pytestmark = pytest.mark.gpu


def device_cache(b, caches=None, table=None):
    """A KVCache holding a batch's arrays (as they are before the new tokens)."""
    k, v, ks, vs = caches if caches is not None else (b.k, b.v, b.ks, b.vs)
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    codes = [t(a).view(torch.float8_e4m3fn) if b.quantised else t(a) for a in (k, v)]
    return qsa.KVCache(*codes, t(b.table if table is None else table), t(ks), t(vs))


def _bits(t):
    return (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16)).cpu().numpy()


def check(cache, want):
    st = qsa.get_device_status()
    assert st == qsa.QSA_OK, qsa.status_string(st)
    k, v, ks, vs = want
    view = (lambda a: a) if k.dtype == np.uint8 else (lambda a: a.view(np.int16))
    np.testing.assert_array_equal(_bits(cache.k), view(k))
    np.testing.assert_array_equal(_bits(cache.v), view(v))
    if ks is not None:
        np.testing.assert_array_equal(cache.k_scale.cpu().numpy(), ks)
        np.testing.assert_array_equal(cache.v_scale.cpu().numpy(), vs)


def on_gpu(b):
    fused = torch.from_numpy(b.fused).cuda()
    return (fused[:, :b.hq], fused[:, b.hq:b.hq + b.hkv], fused[:, b.hq + b.hkv:],
            torch.from_numpy(b.seq_start).cuda(), torch.from_numpy(b.pos_start).cuda())


SHAPES = [(128, 1, 8), (128, 3, 16), (128, 8, 128), (256, 2, 64), (256, 1, 256), (256, 5, 32)]


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("D,hkv,page", SHAPES)
@pytest.mark.parametrize("lens", BATCHES.values(), ids=BATCHES)
def test_store_and_load(lens, D, hkv, page, quantised):
    b = Batch(5, lens, hkv=hkv, group=1, head_dim=D, page=page, quantised=quantised)
    cache = device_cache(b)
    _, k, v, ss, ps = on_gpu(b)
    qsa.kv_store(k, v, ss, ps, cache)
    want = b.stored()
    check(cache, want)
    # all tokens of each request read back: rows of whole requests, then two more
    n = np.array([c for _, c in lens])
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    zero = np.zeros(len(lens), np.int32)
    rows = int(starts[-1]) + 2
    wide = torch.full((rows, 2 * hkv + 1, D), 7.0, dtype=torch.float16, device="cuda")
    gk, gv = wide[:, :hkv], wide[:, hkv + 1:]
    qsa.kv_load(torch.from_numpy(starts).cuda(), torch.from_numpy(zero).cuda(), rows, cache, out_k=gk, out_v=gv)
    assert qsa.get_device_status() == qsa.QSA_OK
    for got, c, s in ((gk, want[0], want[2]), (gv, want[1], want[3])):
        ref = O.load(rows, starts, zero, b.table, c, s)
        ref[starts[-1]:] = 7.0                                            # rows of no request
        np.testing.assert_array_equal(got.cpu().numpy().astype(np.float64), ref)
    assert torch.all(wide[:, hkv] == 7.0)                                 # between the two slices


def test_every_size_and_ties_quantise_exactly():
    """Vectors of every scale, values on the borders between two codes."""
    rng = np.random.default_rng(6)
    D, T = 128, 600
    size = 2.0 ** rng.uniform(-26, 16, (T, 1))
    x = np.clip(rng.standard_normal((T, D)) * size, -65504, 65504).astype(np.float16)
    v = O.e4m3_values()[:127]
    ties = ((v[:-1] + v[1:]) / 2)[None, :] * 2.0 ** rng.integers(-14, 8, (T, 1))
    x[::2, :126] = ties[::2].astype(np.float16)
    x[1::2, 126] = np.where(np.arange(T // 2) % 3 == 0, 65504.0, x[1::2, 126])
    x[7], x[9, 3], x[11, 5], x[13] = 0.0, np.inf, -np.inf, -0.0
    x[15, 4] = np.nan
    lens = [(T, T)]
    b = Batch(7, lens, hkv=1, group=1, head_dim=D, page=64, quantised=True, pad_rows=0)
    b.k_new, b.v_new = x[:, None], x[::-1, None].copy()
    cache = device_cache(b)
    qsa.kv_store(torch.from_numpy(b.k_new).cuda(), torch.from_numpy(b.v_new).cuda(),
                 torch.from_numpy(b.seq_start).cuda(), torch.from_numpy(b.pos_start).cuda(), cache)
    check(cache, b.stored())


@pytest.mark.parametrize("quantised", [False, True])
def test_bad_pages_and_requests_are_flagged_and_skipped(quantised):
    lens = [(6, 40), (5, 5), (4, 30)]
    b = Batch(8, lens, hkv=2, group=1, head_dim=256, page=8, quantised=quantised)
    table = b.table.copy()
    table[0, 4] = b.num_pages + 3                                         # tokens 32 .. 39 of request 0
    cache = device_cache(b, table=table)
    _, k, v, ss, ps = on_gpu(b)
    qsa.kv_store(k, v, ss, ps, cache)
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE
    b.table = table
    want = b.stored()
    check(cache, want)
    gk, gv = qsa.kv_load(ss, ps, b.T, cache, out_k=torch.full_like(k, 7.0).contiguous())
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE
    assert torch.all(gk[:6] == 0) and torch.all(gv[:6] == 0)
    assert torch.all(gk[15:] == 7.0)
    # a negative position, a request past the block table, decreasing starts
    for pos, starts in (([-1, 0, 26], b.seq_start), ([34, 0, b.max_pages * 8], b.seq_start),
                        ([34, 0, 26], [0, 6, 4, 15]), ([34, 0, 26], [0, 6, 11, b.T + 1])):
        c2 = device_cache(b)
        bad_ss = torch.tensor(np.asarray(starts), dtype=torch.int32).cuda()
        qsa.kv_store(k, v, bad_ss, torch.tensor(pos, dtype=torch.int32).cuda(), c2)
        assert qsa.get_device_status() in (qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_BAD_PAGE)


def test_store_on_another_stream_and_captured():
    b = Batch(9, [(33, 70), (1, 9)], hkv=2, group=1, head_dim=128, page=16, quantised=True)
    _, k, v, ss, ps = on_gpu(b)
    want = b.stored()
    side = torch.cuda.Stream()
    cache = device_cache(b)
    torch.cuda.synchronize()
    qsa.kv_store(k, v, ss, ps, cache, stream=side)
    side.synchronize()
    check(cache, want)
    gk, gv = qsa.kv_load(ss, ps, b.T, cache, stream=side)                  # allocated here, written there
    side.synchronize()
    ref = O.load(b.T, b.seq_start, b.pos_start, b.table, want[0], want[2])
    n = int(b.seq_start[-1])
    np.testing.assert_array_equal(gk.cpu().numpy()[:n].astype(np.float64), ref[:n])
    cache = device_cache(b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.kv_store(k, v, ss, ps, cache)
    g.replay()
    torch.cuda.synchronize()
    check(cache, want)


def test_binding_refuses():
    b = Batch(10, [(4, 9)], hkv=2, group=2, head_dim=128, page=8, quantised=False)
    cache = device_cache(b)
    q, k, v, ss, ps = on_gpu(b)
    with pytest.raises(TypeError):
        qsa.kv_store(k.float(), v, ss, ps, cache)
    with pytest.raises(TypeError):
        qsa.kv_store(k, v, ss.long(), ps, cache)
    with pytest.raises(ValueError):
        qsa.kv_store(k.cpu(), v, ss, ps, cache)
    with pytest.raises(ValueError):
        qsa.kv_store(q, v, ss, ps, cache)                                  # four heads
    with pytest.raises(ValueError):
        qsa.kv_store(k, v, ss[:1], ps, cache)
    with pytest.raises(ValueError):
        qsa.kv_store(k, v[:3], ss, ps, cache)
    with pytest.raises(qsa.QSAError):
        odd = torch.zeros(4, 2 * 128 + 4, dtype=torch.float16, device="cuda")[:, :256].view(4, 2, 128)
        qsa.kv_store(odd, v[:4], ss, ps, cache)                            # row stride not a multiple of 8
    with pytest.raises(ValueError):
        qsa.KVCache(cache.k, cache.v, cache.block_table, k_scale=torch.zeros(1, dtype=torch.uint8, device="cuda"))
