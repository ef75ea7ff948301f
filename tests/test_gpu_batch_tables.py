"""GPU: batch_tables against the oracle, number for number."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from oracle import batch_tables as O

pytestmark = pytest.mark.gpu


def t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(seed, n, new_max, ctx_max, P, extra_pages=1):
    """Lengths, a block table with the pages that are in use, a shuffled free list."""
    rng = np.random.default_rng(seed)
    new = rng.integers(0, new_max + 1, n).astype(np.int32)
    ctx = rng.integers(0, ctx_max + 1, n).astype(np.int32)
    have, need = -(-ctx // P), -(-(ctx + new) // P)
    max_pages = int(need.max(initial=0)) + extra_pages
    perm = rng.permutation(int(need.sum()) + 9).astype(np.int32)
    table = np.full((n, max_pages), -1, np.int32)
    at = 0
    for b in range(n):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    return new, ctx, table, perm[at:], int((need - have).sum())


def run(new, ctx, rows, P, table, free, count, batch=None):
    tt, fl = t(table), t(free)
    batch = batch or qsa.Batch.empty(len(new), rows, "cuda")
    qsa.batch_tables(t(new), t(ctx), fl, t(np.array([count], np.int32)), tt, P, batch)
    got = {name: getattr(batch, name).cpu().numpy() for name in qsa.Batch._NAMES}
    got["block_table"] = tt.cpu().numpy()
    np.testing.assert_array_equal(fl.cpu().numpy(), free)
    return got


def check(got, want):
    for name in want:
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)


SIZES = [(1, 1, 0, 8), (1, 1, 127, 128), (1, 5000, 100, 8), (2, 3, 9, 16), (64, 1, 3000, 64), (33, 700, 900, 32),
         (1023, 3, 50, 16), (1025, 9, 50, 8), (9000, 2, 300, 256), (65535, 1, 40, 16), (5, 0, 100, 16)]


@pytest.mark.parametrize("n,new_max,ctx_max,P", SIZES)
def test_matches_the_oracle(n, new_max, ctx_max, P):
    new, ctx, table, free, fresh = make(70, n, new_max, ctx_max, P)
    total = int(new.sum())
    # all fit; rows end in the middle; pages do; nothing does
    for rows, count in ((total + 37, fresh + 3), (total, fresh), (total * 2 // 3, fresh + 9), (total + 5, fresh // 2),
                        (total, max(fresh - 1, 0)), (0, 0)):
        want, bad = O.tables(new, ctx, rows, P, table, free, count)
        assert not bad
        check(run(new, ctx, rows, P, table, free, count), want)
        assert qsa.get_device_status() == qsa.QSA_OK


def test_no_requests():
    e = np.zeros(0, np.int32)
    got = run(e, e, 5, 16, np.zeros((0, 3), np.int32), np.arange(4, dtype=np.int32), 4)
    assert got["seq_start"].tolist() == [0] and got["state"].tolist() == [0, 4, 0] and got["slot"].tolist() == [-1] * 5
    assert got["row_req"].tolist() == [0] * 5


def test_bad_lengths_and_lists():
    new, ctx, table, free, fresh = make(71, 40, 30, 200, 16)
    for b, (x, y) in {3: (-1, 5), 9: (4, -3), 20: (2 ** 31 - 1, 2 ** 31 - 1), 39: (0, table.shape[1] * 16 + 1),
                      11: (table.shape[1] * 16, 1)}.items():
        new[b], ctx[b] = x, y
    for count in (fresh, len(free) + 100, -4, fresh // 3):
        want, bad = O.tables(new, ctx, 700, 16, table, free, count)
        assert bad
        check(run(new, ctx, 700, 16, table, free, count), want)
        assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG


def test_bad_pages():
    """Pages without a place in 31 bits give slot -1, reported; the rest is right."""
    new, ctx, table, free, fresh = make(72, 4, 20, 100, 16)
    new[:], ctx[:] = 3, 5
    table[1, 0], table[2, 0] = -1, 2 ** 27
    got = run(new, ctx, 12, 16, table, free, len(free))
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE
    assert got["slot"].tolist()[3:9] == [-1] * 6
    for r in (0, 11):
        b, tok = r // 3, 5 + r % 3
        assert got["slot"][r] == table[b, 0] * 16 + tok


def test_a_page_just_inside_31_bits():
    new, ctx = np.array([2], np.int32), np.array([14], np.int32)
    table = np.array([[2 ** 27 - 1, -1]], np.int32)
    got = run(new, ctx, 2, 16, table, np.array([3], np.int32), 1)
    assert qsa.get_device_status() == qsa.QSA_OK
    assert got["slot"].tolist() == [2 ** 31 - 2, 2 ** 31 - 1]


def test_maps_left_out():
    """Optional arrays may be NULL, here through the C entry."""
    import ctypes
    new, ctx, table, free, fresh = make(73, 20, 5, 60, 8)
    want, _ = O.tables(new, ctx, 200, 8, table, free, fresh)
    b = qsa.Batch.empty(20, 200, "cuda")
    for keep in (set(), {"row_token"}, {"slot"}, {"row_req", "row_visible"}):
        for name in qsa.Batch._NAMES:
            getattr(b, name).fill_(-7)
        c = qsa.BatchC(*(getattr(b, n).data_ptr() if n in keep | {"seq_start", "pos_start", "state"} else None
                         for n in qsa.Batch._NAMES))
        tt = t(table)
        a = [t(x) for x in (new, ctx, free, np.array([fresh], np.int32))]
        st = qsa.load().qsa_batch_tables(a[0].data_ptr(), a[1].data_ptr(), 20, 200, 8, tt.data_ptr(), table.shape[1],
                                         a[2].data_ptr(), len(free), a[3].data_ptr(), ctypes.byref(c), None)
        assert st == qsa.QSA_OK and qsa.get_device_status() == qsa.QSA_OK
        np.testing.assert_array_equal(tt.cpu().numpy(), want["block_table"])
        for name in qsa.Batch._NAMES:
            got = getattr(b, name).cpu().numpy()
            np.testing.assert_array_equal(got, want[name] if name in keep | {"seq_start", "pos_start", "state"}
                                          else np.full_like(got, -7))


@pytest.mark.parametrize("n,P", [(50, 16), (3000, 8)])
def test_steps_that_go_on_from_their_own_results(n, P):
    """total_len over ctx_len and the list's count in place: decode steps of a captured graph."""
    new, ctx, table, free, _ = make(74, n, 1, 40, P, extra_pages=6)
    rng = np.random.default_rng(1)
    free = (int(table.max(initial=0)) + 1 + rng.permutation(4 * n)).astype(np.int32)
    e = qsa.Batch.empty(n, 2 * n, "cuda")
    lens = t(ctx)
    e = qsa.Batch(e.seq_start, e.pos_start, lens, e.row_req, e.row_token, e.row_visible, e.slot, e.state)
    nt, tt, fl = t(new), t(table), t(free)
    e.state.copy_(torch.tensor([0, len(free), 0], dtype=torch.int32))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qsa.batch_tables(nt, lens, fl, e.state[1:2], tt, P, e)
    left = len(free)
    for step in range(12):
        new = rng.integers(0, 3, n).astype(np.int32)
        nt.copy_(torch.from_numpy(new))
        g.replay()
        want, bad = O.tables(new, ctx, 2 * n, P, table, free, left)
        assert not bad
        got = {name: getattr(e, name).cpu().numpy() for name in qsa.Batch._NAMES}
        got["block_table"] = tt.cpu().numpy()
        check(got, want)
        table, ctx, left = want["block_table"], want["total_len"], int(want["state"][1])
    assert qsa.get_device_status() == qsa.QSA_OK


def test_refusals_in_python():
    b = qsa.Batch.empty(3, 8, "cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(new_len=i(3), ctx_len=i(3), free_pages=i(5), free_count=i(1), block_table=i(3, 4), page_tokens=16, batch=b)
    for kw, err in [(dict(new_len=i(2)), ValueError), (dict(ctx_len=i(3).long()), TypeError), (dict(free_count=i(2)), ValueError),
                    (dict(block_table=i(2, 4)), ValueError), (dict(block_table=i(12)), ValueError),
                    (dict(new_len=i(6)[::2]), ValueError), (dict(free_pages=i(5).cpu()), ValueError),
                    (dict(page_tokens=24), qsa.QSAError)]:
        with pytest.raises(err):
            qsa.batch_tables(**{**good, **kw})
    assert qsa.batch_tables(**good) is b
    with pytest.raises(AttributeError):
        b.slot = i(8)
    with pytest.raises(ValueError):
        qsa.Batch(i(4), i(3), i(3), i(8), i(8), i(8), i(7), i(3))
    assert qsa.get_device_status() == qsa.QSA_OK
