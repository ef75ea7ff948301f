"""CPU: the K/V cache oracle against independent definitions."""
import numpy as np
import pytest
import torch

from kv_util import Batch
from oracle import kv_cache as O


def test_encode_agrees_with_the_format():
    v = O.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, t)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 0.01,
                        (v[:126] + v[1:127]) / 2, -(v[:126] + v[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]])
    want = torch.from_numpy(y.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(O.encode(y.astype(np.float32).astype(np.float64)), want)


@pytest.mark.parametrize("size", [2.0 ** -24, 1e-4, 0.0136, 0.0137, 0.3, 1.0, 447.0, 448.0, 449.0, 3e4, 65504.0])
def test_stored_values_are_fp16_numbers_near_the_input(size):
    rng = np.random.default_rng(1)
    x = (rng.uniform(-1, 1, (64, 128)) * size).astype(np.float16)
    x[:, 0] = np.float16(size)
    code, scale = O.quantise(x)
    e = scale.astype(int) - 127
    assert e.min() >= -15 and e.max() <= 8
    y = O.dequantise(code, scale)
    assert np.all(np.isfinite(y))
    np.testing.assert_array_equal(y.astype(np.float16).astype(np.float64), y)
    err = np.abs(y - x.astype(np.float64))
    assert np.all(err <= np.maximum(np.abs(x.astype(np.float64)) / 16, 2.0 ** (e[:, None] - 10)))


def test_scale_is_the_least_that_holds_the_vector():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((500, 128)) * 2.0 ** rng.uniform(-12, 10, (500, 1))).astype(np.float16)
    x = x[np.isfinite(x).all(-1)]
    _, scale = O.quantise(x)
    a, e = np.abs(x.astype(np.float64)).max(-1), scale.astype(int) - 127
    assert np.all((a <= 448 * 2.0 ** e) | (e == 8))
    assert np.all((a > 448 * 2.0 ** (e - 1)) | (e == -15))


def test_attention_of_a_constant_cache_is_the_mean():
    b = Batch(3, [(4, 20)], hkv=1, group=2, head_dim=128, page=8, quantised=False)
    k, v, _, _ = b.stored()
    k = np.zeros_like(k)                                  # equal scores
    out, mag = O.attention(b.q, b.seq_start, b.pos_start, b.table, k, v, window=5)
    rows = O.load(20, [0, 20], [0], b.table, v)
    for i in range(4):
        np.testing.assert_allclose(out[i, 1], rows[16 + i - 4:16 + i + 1, 0].mean(0), rtol=1e-12, atol=1e-12)
    assert np.isnan(out[4:]).all() and np.all(mag[:4] >= np.abs(out[:4]))
