"""GPU: block_attention against the 64-bit oracle (kv_util.tolerance)."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import BATCHES, Batch, tolerance
from oracle import block_attention as O
from test_gpu_kv_cache import device_cache, on_gpu

pytestmark = pytest.mark.gpu

# head_dim, KV heads, query heads per KV head, page tokens
SHAPES = [(128, 2, 1, 8), (128, 1, 5, 128), (128, 3, 16, 16), (256, 2, 12, 64), (256, 1, 4, 256), (256, 1, 1, 32)]


def positions(b):
    """Position of every row, -1 behind the last request."""
    pos = np.full(b.T, -1)
    for r in range(len(b.lens)):
        s0, s1 = b.seq_start[r], b.seq_start[r + 1]
        pos[s0:s1] = b.pos_start[r] + np.arange(s1 - s0)
    return pos


def select(b, k, seed, none=0.2, rows_alike=False):
    """Visible blocks in any order, some twice, some -1; now and then a row of
    nothing but -1.  rows_alike: neighbouring rows share most of their blocks."""
    rng = np.random.default_rng(seed)
    sel = np.full((b.T, b.hkv, k), -1, np.int32)
    old = None
    for r, p in enumerate(positions(b)):
        if p < 0:
            sel[r] = rng.integers(-9, 1 << 30, (b.hkv, k))              # rows of no request: anything
            continue
        x = rng.integers(0, p // 128 + 1, (b.hkv, k))
        if rows_alike and old is not None and old.max(initial=0) <= p // 128:
            x = np.where(rng.random(x.shape) < 0.8, old, x)
        old = x
        sel[r] = np.where(rng.random(x.shape) < none, -1, x)
        if rng.random() < 0.1:
            sel[r] = -1
    return sel


def hide(b, caches, sel, recent):
    """Copies of the caches with NaN in every slot that no row attends, and of the
    block table with -1 for every page that no row attends."""
    k, v, ks, vs = (None if a is None else a.copy() for a in caches)
    table = b.table.copy()
    seen = np.zeros((len(b.lens), b.max_pages * b.P, b.hkv), bool)
    pos = positions(b)
    for r in range(len(b.lens)):
        for row in range(b.seq_start[r], b.seq_start[r + 1]):
            for g in range(b.hkv):
                seen[r, O.attended(sel[row, g], pos[row], recent), g] = True
        for pg in range(b.max_pages):
            here = seen[r, pg * b.P:(pg + 1) * b.P]
            if not here.any():
                table[r, pg] = -1
            else:
                for a in (k, v):
                    a[b.table[r, pg]][~here] = 0x7F if b.quantised else np.nan
    return (k, v, ks, vs), table


def attend(b, caches, sel, recent=0, scale=None, table=None, **kw):
    cache = device_cache(b, caches, table)
    q, _, _, ss, ps = on_gpu(b)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    qsa.block_attention(q, torch.from_numpy(sel).cuda(), ss, ps, cache, recent=recent, scale=scale, out=out, **kw)
    return out


def check(b, got, caches, sel, recent=0, scale=None, vmax=6.0):
    k, v, ks, vs = caches
    want, mag = O.attention(b.q, sel, b.seq_start, b.pos_start, b.table, k, v, ks, vs, recent, scale)
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
    for i, (k, recent) in enumerate([(3, 0), (2, 1)]):
        sel = select(b, k, 41 + i, rows_alike=i == 1)
        hidden, table = hide(b, caches, sel, recent)
        got = attend(b, hidden, sel, recent, table=table)
        ok()
        check(b, got, caches, sel, recent)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("k,recent", [(1, 0), (1, 1), (0, 1), (0, 3), (5, 2), (16, 1), (40, 0), (300, 100)])
@pytest.mark.parametrize("D,group,page", [(128, 12, 128), (256, 3, 16)])
def test_numbers_of_blocks(k, recent, D, group, page, quantised):
    lens = [(33, 1400), (1, 1700), (2, 640), (1, 1)]
    b = Batch(32, lens, hkv=2, group=group, head_dim=D, page=page, quantised=quantised)
    caches = b.stored()
    sel = select(b, k, 43)
    hidden, table = hide(b, caches, sel, recent)
    got = attend(b, hidden, sel, recent, table=table)
    ok()
    check(b, got, caches, sel, recent)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("lens", [[(1, 1000), (1, 2500), (1, 129)], [(300, 900), (270, 270)]], ids=["step", "prompt"])
def test_every_block_is_dense_attention(lens, quantised):
    """Every block selected: the numbers of chunk_attention, within both roundings."""
    b = Batch(33, lens, hkv=2, group=6, head_dim=128, page=64, quantised=quantised)
    caches = b.stored()
    sel = np.tile(np.random.default_rng(1).permutation(20).astype(np.int32), (b.T, b.hkv, 1))
    sel = np.where(sel * 128 <= positions(b)[:, None, None], sel, -1)
    got = attend(b, caches, sel)
    cache = device_cache(b, caches)
    q, _, _, ss, ps = on_gpu(b)
    dense = qsa.chunk_attention(q, ss, ps, cache)
    ok()
    check(b, got, caches, sel)
    n = int(b.seq_start[-1])
    want, mag = b.attention(caches)
    tol = 2 * tolerance(want[:n], mag[:n], b.lens, 6.0)
    assert np.all(np.abs(got[:n].cpu().numpy().astype(float) - dense[:n].cpu().numpy().astype(float)) <= tol)


def test_rows_that_attend_nothing():
    """Whole units of them, and single ones between others."""
    for lens in ([(1, 700), (1, 5)], [(600, 900)], [(40, 300), (1, 300)]):
        b = Batch(34, lens, hkv=2, group=4, head_dim=128, page=32, quantised=False)
        caches = b.stored()
        sel = select(b, 3, 44, none=0.0)
        for keep in (np.zeros(b.T, bool), np.arange(b.T) % 50 == 7):
            s = np.where(keep[:, None, None], sel, -1)
            hidden, table = hide(b, caches, s, 0)
            got = attend(b, hidden, s, table=table)
            ok()
            check(b, got, caches, s)
            idle = np.flatnonzero(~keep[:int(b.seq_start[-1])])
            assert not got[torch.from_numpy(idle).cuda()].any()


@pytest.mark.parametrize("hkv,group,lens", [(1, 128, [(3, 300), (1, 500)]), (2, 17, [(1, 600), (1, 900)]),
                                            (2, 100, [(5, 400)]), (1, 24, [(1, 40)] * 5), (8, 1, [(500, 800)])])
def test_groups(hkv, group, lens):
    b = Batch(35, lens, hkv=hkv, group=group, head_dim=128, page=16, quantised=False)
    caches = b.stored()
    sel = select(b, 3, 45)
    got = attend(b, caches, sel, 1)
    ok()
    check(b, got, caches, sel, 1)


@pytest.mark.parametrize("lens", [[(1, 700), (1, 300)], [(90, 700), (60, 300)]], ids=["step", "chunk"])
def test_bad_blocks_and_pages(lens):
    b = Batch(36, lens, hkv=2, group=4, head_dim=128, page=64, quantised=False)
    caches = b.stored()
    sel = select(b, 4, 46, none=0.0)
    good = sel.copy()
    n = int(b.seq_start[-1])
    # names that no block has are ignored, and reported
    for row, g, i, c in ((0, 0, 1, -2), (n - 1, 1, 0, 6), (n - 1, 0, 3, 2 ** 31 - 1), (0, 1, 2, -2 ** 31)):
        sel[row, g, i], good[row, g, i] = c, -1
    got = attend(b, caches, sel)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    check(b, got, caches, good)
    # a page outside the cache: zero keys and values, reported
    b.table[0, 3] = b.num_pages
    b.table[1, 0] = -5
    got = attend(b, caches, good, 1)
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE
    check(b, got, caches, good, 1)


@pytest.mark.parametrize("group", [1, 12])
def test_bad_requests(group):
    """Requests that are out of range are skipped, the others served."""
    lens = [(4, 300), (70, 200), (1, 500), (30, 129)]
    b = Batch(37, lens, hkv=2, group=group, head_dim=128, page=32, quantised=False)
    caches = b.stored()
    sel = select(b, 3, 47)
    good_start = b.pos_start.copy()
    b.pos_start[1] = -1
    b.pos_start[3] = b.max_pages * b.P
    got = attend(b, caches, sel, 1)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    want, mag = O.attention(b.q, sel, b.seq_start, good_start, b.table, *caches[:2], recent=1)
    got = got.cpu().numpy().astype(np.float64)
    for r in range(4):
        s = slice(b.seq_start[r], b.seq_start[r + 1])
        if r in (1, 3):
            assert np.all(got[s] == 7.0)
        else:
            assert np.all(np.abs(got[s] - want[s]) <= tolerance(want[s], mag[s], lens, 6.0))


def test_falling_starts():
    """Starts out of order cost only the requests they make impossible."""
    b = Batch(38, [(20, 300), (30, 400)], hkv=1, group=4, head_dim=128, page=32, quantised=False)
    caches = b.stored()
    sel = select(b, 3, 48)
    cache = device_cache(b, caches, np.concatenate([b.table[1:], b.table[:1], b.table[:1]]))
    q, _, _, _, _ = on_gpu(b)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    # rows 20 .. 49 first, then a request from 50 to 0, then rows 0 .. 19
    ss = torch.tensor([20, 50, 0, 20], dtype=torch.int32, device="cuda")
    ps = torch.tensor([370, 0, 280], dtype=torch.int32, device="cuda")
    qsa.block_attention(q, torch.from_numpy(sel).cuda(), ss, ps, cache, out=out)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    check(b, out, caches, sel)


@pytest.mark.parametrize("quantised", [False, True])
def test_large_and_small_scores(quantised):
    b = Batch(39, [(40, 1000), (1, 900)], hkv=1, group=4, head_dim=256, page=16, quantised=quantised)
    k, v, ks, vs = b.stored()
    if not quantised:
        for t in range(0, 960, 100):                       # ever larger keys along the first request
            k[b.table[0, t // 16], t % 16] *= np.float16(1 + t / 200)
    sel = select(b, 5, 49)
    got = attend(b, (k, v, ks, vs), sel, 1, scale=0.5)
    ok()
    # scores of tens: their FP32 sums are off by head_dim * 2^-24 * scale * sum |q k|, 2^-7.5 at
    # |q| |k| * scale of 360, which moves a weight by 2^-7.5 of itself at most, twice
    want, mag = O.attention(b.q, sel, b.seq_start, b.pos_start, b.table, k, v, ks, vs, 1, 0.5)
    n = 41
    off = np.abs(got[:n].cpu().numpy().astype(float) - want[:n])
    assert np.all(off <= 2.0 ** -11 * np.abs(want[:n]) + 2.0 ** -6 * mag[:n] + 2.0 ** -14)


def test_many_requests_and_heads():
    rng = np.random.default_rng(5)
    lens = [(int(n), int(n + rng.integers(0, 300))) for n in rng.integers(0, 4, 1300)]
    b = Batch(40, lens, hkv=2, group=2, head_dim=128, page=64, quantised=False)
    caches = b.stored()
    sel = select(b, 2, 50)
    got = attend(b, caches, sel, 1)
    ok()
    check(b, got, caches, sel, 1)
    # the same requests as one prompt each of a longer batch
    lens = [(200, 400)] * 9 + [(0, 3)] * 60 + [(130, 130)] * 3
    b = Batch(41, lens, hkv=3, group=3, head_dim=128, page=8, quantised=False)
    caches = b.stored()
    sel = select(b, 2, 51, rows_alike=True)
    got = attend(b, caches, sel)
    ok()
    check(b, got, caches, sel)


@pytest.mark.parametrize("lens", [[(1, 700)] * 6, [(90, 700), (60, 300)]], ids=["step", "chunk"])
def test_graphs_and_streams(lens):
    """Two graphs with workspaces of their own replayed at once on two streams, and
    an eager call on a third, with the lengths and blocks changed in place."""
    b = Batch(42, lens, hkv=2, group=4, head_dim=128, page=32, quantised=False)
    caches = b.stored()
    cache = device_cache(b, caches)
    q, _, _, ss, ps = on_gpu(b)
    sels = [select(b, 3, 52 + i) for i in range(3)]
    dev = [torch.from_numpy(s).cuda() for s in sels]
    outs = [torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda") for _ in range(3)]
    graphs = []
    for i in range(2):
        ws = qsa.alloc_block_attention_workspace(cache, b.T, b.hq, 3, 1)
        args = dict(recent=1, out=outs[i], ws=ws)
        qsa.block_attention(q, dev[i], ss, ps, cache, **args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qsa.block_attention(q, dev[i], ss, ps, cache, **args)
        graphs.append((g, ws))
    dev[0].copy_(torch.from_numpy(sels[1]))
    dev[1].copy_(torch.from_numpy(sels[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i][0].replay()
        qsa.block_attention(q, dev[2], ss, ps, cache, recent=1, out=outs[2], stream=streams[2])
    torch.cuda.synchronize()
    ok()
    for i, s in enumerate((1, 0, 2)):
        check(b, outs[i], caches, sels[s], 1)


def test_results_are_repeatable():
    b = Batch(43, [(1, 2000), (130, 900), (1, 128)], hkv=2, group=8, head_dim=128, page=64, quantised=True)
    caches = b.stored()
    sel = select(b, 6, 55)
    first = attend(b, caches, sel, 1)
    for _ in range(5):
        assert torch.equal(first, attend(b, caches, sel, 1))


def test_refusals_in_python():
    b = Batch(44, [(2, 40)], hkv=2, group=2, head_dim=128, page=16, quantised=False)
    cache = device_cache(b, b.stored())
    q, _, _, ss, ps = on_gpu(b)
    sel = torch.zeros(b.T, 2, 3, dtype=torch.int32, device="cuda")
    call = lambda **kw: qsa.block_attention(**{**dict(q=q, sel=sel, seq_start=ss, pos_start=ps, cache=cache), **kw})  # noqa: E731
    for kw, err in [(dict(q=q.float()), TypeError), (dict(sel=sel.long()), TypeError), (dict(sel=sel[:1]), ValueError),
                    (dict(sel=sel.cpu()), ValueError), (dict(sel=sel[..., :2]), ValueError), (dict(sel=sel[:, :1]), ValueError),
                    (dict(out=q[:, :2].contiguous()), ValueError), (dict(recent=-1), qsa.QSAError), (dict(scale=-1.0), qsa.QSAError),
                    (dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")), qsa.QSAError)]:
        with pytest.raises(err):
            call(**kw)
    assert call().shape == q.shape
    ok()


# Selections taken straight, a cluster of CTAs to a row and KV head while those are
# few (8, 4, 2 and 1), several rows to a CTA when they are many; 32 blocks at most.
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("reqs,hkv,group,k,recent", [(1, 1, 1, 3, 0), (1, 2, 12, 16, 1), (3, 8, 4, 5, 0), (9, 5, 16, 31, 1),
                                                     (40, 2, 3, 16, 2), (70, 3, 9, 32, 0), (2, 1, 7, 0, 32), (5, 2, 2, 33, 0)])
def test_single_tokens(reqs, hkv, group, k, recent, D, quantised):
    rng = np.random.default_rng(reqs)
    lens = [(1, int(c)) for c in rng.integers(1, 2600 if reqs < 20 else 900, reqs)]
    b = Batch(45, lens, hkv=hkv, group=group, head_dim=D, page=32, quantised=quantised)
    caches = b.stored()
    sel = select(b, k, 56)
    hidden, table = hide(b, caches, sel, recent)
    got = attend(b, hidden, sel, recent, table=table)
    ok()
    check(b, got, caches, sel, recent)


@pytest.mark.parametrize("reqs", [3, 200])
def test_single_tokens_of_a_changing_batch(reqs):
    """Empty requests, padding, starts that fall and requests out of range among single tokens."""
    rng = np.random.default_rng(7)
    lens = [(int(rng.random() < 0.7), int(rng.integers(1, 700))) for _ in range(reqs)]
    b = Batch(46, lens, hkv=2, group=3, head_dim=128, page=64, quantised=False, pad_rows=reqs - sum(n for n, _ in lens))
    caches = b.stored()
    sel = select(b, 4, 57)
    got = attend(b, caches, sel, 1)
    ok()
    check(b, got, caches, sel, 1)
    # the same rows in two runs, the later one first, and a request past the block table
    n = int(b.seq_start[-1])
    order = [i for i in range(reqs) if lens[i][0]]
    order = order[len(order) // 2:] + order[:len(order) // 2]
    starts = [int(b.seq_start[i]) for i in order]
    ss = torch.tensor(starts + [starts[-1] + 1], dtype=torch.int32, device="cuda")
    ps = torch.tensor(b.pos_start[order], device="cuda")
    cache = device_cache(b, caches, np.concatenate([b.table[order], b.table[:1]]))
    q, _, _, _, _ = on_gpu(b)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    qsa.block_attention(q, torch.from_numpy(sel).cuda(), ss, ps, cache, recent=1, out=out)
    k, v, ks, vs = caches
    want, mag = O.attention(b.q, sel, b.seq_start, b.pos_start, b.table, k, v, ks, vs, 1)
    got = out.cpu().numpy().astype(np.float64)
    assert qsa.get_device_status() == (qsa.QSA_ERR_INVALID_ARG if len(order) > 1 else qsa.QSA_OK)
    # where the starts fall, the request before has no rows (its end lies before its start)
    lost = [s for s, e in zip(starts, starts[1:] + [starts[-1] + 1]) if e <= s]
    rows = [r for r in range(n) if r not in lost]
    assert np.all(np.abs(got[rows] - want[rows]) <= tolerance(want[rows], mag[rows], lens, 6.0))
    assert np.all(got[lost] == 7.0) and np.all(got[n:] == 7.0)
