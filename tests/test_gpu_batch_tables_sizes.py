"""GPU: batch_tables on both sides of the sizes at which it changes its launch: one CTA
or a cluster, starts and positions in shared memory (asked for, or not) or from global."""
import pytest

from block_sparse_attention_select_gb300 import qsa
from oracle import batch_tables as O
from test_gpu_batch_tables import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2047, 2048, 2049, 3071, 3073, 5000, 8190, 8191, 8192])
def test_numbers_of_requests(n):
    new, ctx, table, free, fresh = make(75, n, 3, 60, 16)
    total = int(new.sum())
    for rows, count in ((total + 37, fresh + 3), (total * 2 // 3, fresh + 9), (total + 5, fresh // 2)):
        want, bad = O.tables(new, ctx, rows, 16, table, free, count)
        assert not bad
        check(run(new, ctx, rows, 16, table, free, count), want)
        assert qsa.get_device_status() == qsa.QSA_OK


@pytest.mark.parametrize("rows", [8191, 8192, 8193])
@pytest.mark.parametrize("n,new_max", [(3, 5400), (700, 23), (2048, 7)])
def test_numbers_of_rows(n, new_max, rows):
    new, ctx, table, free, fresh = make(76, n, new_max, 100, 32)
    want, bad = O.tables(new, ctx, rows, 32, table, free, fresh)
    assert not bad
    check(run(new, ctx, rows, 32, table, free, fresh), want)
    assert qsa.get_device_status() == qsa.QSA_OK
