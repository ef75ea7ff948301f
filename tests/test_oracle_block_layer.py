"""The oracles of batch tables, rotary positions and block attention against
hand-made examples and independent forms."""
import numpy as np
import pytest

from oracle import batch_tables as BT
from oracle import block_attention as BA
from oracle import kv_cache as KV
from oracle import rotary as R


def test_tables_by_hand():
    table = np.full((3, 4), -1, np.int32)
    table[0, 0], table[1, :2] = 5, (6, 7)
    out, bad = BT.tables([3, 1, 9], [7, 16, 0], 20, 8, table, np.array([9, 8, 4, 3, 2], np.int32), 5)
    assert not bad
    assert out["seq_start"].tolist() == [0, 3, 4, 13] and out["state"].tolist() == [13, 1, 3]
    assert out["block_table"].tolist() == [[5, 2, -1, -1], [6, 7, 3, -1], [4, 8, -1, -1]]
    assert out["slot"][:5].tolist() == [47, 16, 17, 24, 32] and out["slot"][12:].tolist() == [64] + [-1] * 7
    assert out["row_token"][:4].tolist() == [7, 8, 9, 16] and out["row_visible"][:4].tolist() == [2, 2, 2, 4]
    out, _ = BT.tables([3, 1, 9], [7, 16, 0], 20, 8, table, np.array([9, 8], np.int32), 2)
    assert out["state"].tolist() == [4, 0, 2] and out["seq_start"].tolist() == [0, 3, 4, 4]
    assert out["total_len"].tolist() == [10, 17, 0]


def test_rotary_keeps_relative_positions():
    """q at p + d and k at p have the same product for every p."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 1, 1, 64))
    for kind in (None, "linear", "base", "parts"):
        f = R.frequencies(32, 10000.0, kind, 4.0, 512)
        for inter in (False, True):
            dots = [(R.rotate(q, np.array([p + 11]), f, 16, inter) * R.rotate(k, np.array([p]), f, 16, inter)).sum()
                    for p in (0, 5, 1000)]
            np.testing.assert_allclose(dots, dots[0], rtol=0, atol=1e-9)
    f = R.frequencies(4, 100.0)
    np.testing.assert_allclose(f, [1.0, 0.1])
    y = R.rotate(np.array([[[1.0, 0, 0, 2.0]]]), np.array([3]), f, 0, False)
    np.testing.assert_allclose(y[0, 0], [np.cos(3), -2 * np.sin(0.3), np.sin(3), 2 * np.cos(0.3)])


def test_scalings():
    f = R.frequencies(64, 10000.0)
    g = R.frequencies(64, 10000.0, "parts", 8.0, 4096)
    turns = 4096 * f / (2 * np.pi)
    np.testing.assert_allclose(g[turns > 32], f[turns > 32])
    np.testing.assert_allclose(g[turns < 1], f[turns < 1] / 8)
    base = R.frequencies(64, 10000.0, "base", 8.0)
    np.testing.assert_allclose([base[0], base[-1]], [1.0, f[-1] / 8])        # the slowest pair is slowed by the factor
    np.testing.assert_allclose(R.frequencies(64, 10000.0, "linear", 8.0), f / 8)


@pytest.mark.parametrize("recent", [0, 1, 2, 50])
def test_all_blocks_are_dense_attention(recent):
    rng = np.random.default_rng(4)
    q = rng.standard_normal((5, 4, 128)).astype(np.float16)
    k, v = rng.standard_normal((2, 30, 16, 2, 128)).astype(np.float16)
    args = (np.array([0, 5]), np.array([395]), rng.permutation(30)[None], k, v)
    sel = np.broadcast_to(np.array([3, 0, 2, 1, 2, -1]), (5, 2, 6))
    a, b = BA.attention(q, sel, *args, recent=recent), KV.attention(q, *args)
    np.testing.assert_allclose(a[0], b[0], atol=1e-12)
    np.testing.assert_allclose(a[1], b[1], atol=1e-12)


def test_attended():
    assert BA.attended([-1, 5], 300, 0).size == 0                              # nothing, and a block not there yet
    assert BA.attended([2, 2, 0], 300, 0).tolist() == list(range(128)) + list(range(256, 301))
    assert BA.attended([], 300, 2).tolist() == list(range(128, 301))
    assert BA.attended([], 3, 9).tolist() == [0, 1, 2, 3]
