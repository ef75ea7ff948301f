"""GPU: the K/V cache calls on batches whose seq_start falls or leaves the rows:
each well-formed request is served by all of them, no other slot or row is
touched."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import Batch, tolerance
from oracle import kv_cache as O
from test_gpu_kv_cache import check, device_cache, on_gpu

pytestmark = pytest.mark.gpu

LENS = [(10, 90), (4, 44), (6, 50), (3, 61)]
FIRST = [80, 40, 44, 58]
# seq_start, pos_start, the requests that are served (no two claim a row)
CASES = {
    "falls_to_empty_ones": ([0, 10, 3, 3, 3], FIRST, [0]),
    "leaves_the_rows": ([0, 5, 1000, 5, 9], FIRST, [0, 3]),
    "falls_in_front": ([7, 3, 9, 12, 14], FIRST, [1, 2, 3]),
    "starts_below_zero": ([-3, 4, 8, 8, 10], FIRST, [1, 3]),
    "ends_past_the_rows": ([0, 6, 10, 14, 27], FIRST, [0, 1, 2]),
    "starts_at_the_smallest_number": ([-2 ** 31, 4, 8, 8, 10], FIRST, [1, 3]),
    "falls_to_the_smallest_number": ([0, 10, -2 ** 31, 14, 20], FIRST, [0, 3]),
    "falls_at_the_end": ([0, 10, 14, 20, 2], FIRST, [0, 1, 2]),
    "rises_far_and_returns": ([12, 1 << 30, 12, 12, 15], FIRST, [3]),
    "negative_position": ([0, 10, 14, 20, 23], [80, -1, 44, 58], [0, 2, 3]),
    "past_the_table": ([0, 10, 14, 20, 23], [80, 40, 1 << 30, 58], [0, 1, 3]),
}


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("starts,first,good", CASES.values(), ids=CASES)
def test_well_formed_requests_are_served_and_nothing_else(starts, first, good, quantised):
    b = Batch(61, LENS, hkv=2, group=2, head_dim=128, page=16, quantised=quantised)
    assert b.T == 26
    cache = device_cache(b)
    q, k, v, _, _ = on_gpu(b)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ss, ps = i32(starts), i32(first)
    one = [(np.array(starts[i:i + 2]), np.array(first[i:i + 1]), b.table[i:i + 1]) for i in good]
    want = (b.k, b.v, b.ks, b.vs)
    for a in one:
        kk, ks = O.store(b.k_new, *a, want[0], want[2])
        vv, vs = O.store(b.v_new, *a, want[1], want[3])
        want = kk, vv, ks, vs
    qsa.kv_store(k, v, ss, ps, cache)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    check(cache, want)

    gk, gv = (torch.full_like(x, 7.0).contiguous() for x in (k, v))
    qsa.kv_load(ss, ps, b.T, cache, out_k=gk, out_v=gv)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    qsa.chunk_attention(q, ss, ps, cache, out=out)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    taken = np.zeros(b.T, bool)
    for a in one:
        rows = slice(int(a[0][0]), int(a[0][1]))
        taken[rows] = True
        for got, c, s in ((gk, want[0], want[2]), (gv, want[1], want[3])):
            np.testing.assert_array_equal(got.cpu().numpy()[rows].astype(np.float64), O.load(b.T, *a, c, s)[rows])
        ref, mag = O.attention(b.q, *a, *want)
        off = np.abs(out.cpu().numpy()[rows].astype(np.float64) - ref[rows])
        assert np.all(off <= tolerance(ref[rows], mag[rows], LENS, 6.0))
    for got in (gk, gv, out):
        assert np.all(got.cpu().numpy()[~taken] == 7.0)


def test_padding_behind_many_requests():
    """Rows behind the last of 700 requests, in CTAs of their own and in shared ones."""
    lens = [(1 + i % 3, 2 + i % 5 + i % 3) for i in range(700)]
    b = Batch(62, lens, hkv=1, group=1, head_dim=128, page=8, quantised=False, pad_rows=900)
    cache = device_cache(b)
    _, k, v, ss, ps = on_gpu(b)
    qsa.kv_store(k, v, ss, ps, cache)
    check(cache, b.stored())


def test_a_cache_keeps_its_tensors():
    """Another tensor put in a cache's attribute would not reach the kernels."""
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for quantised in (False, True):
        cache = qsa.KVCache.empty(3, 16, 2, 128, table, quantised=quantised)
        for name in ("k", "v", "block_table", "k_scale", "v_scale"):
            before = getattr(cache, name)
            with pytest.raises(AttributeError):
                setattr(cache, name, torch.zeros(5, device="cuda"))
            assert getattr(cache, name) is before
