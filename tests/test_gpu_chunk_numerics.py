"""GPU: chunk_attention where its numbers are far from ordinary ones, against 64
bits."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from test_gpu_chunk_attention import reference64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(k, v, quantised, page=32):
    """A cache of one request that holds the rows k, v [tokens, 1, D]."""
    n, _, D = k.shape
    pages = -(-n // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    cache = qsa.KVCache.empty(pages, page, 1, D, table, quantised=quantised)
    qsa.kv_store(k, v, i32([0, n]), i32([0]), cache)
    return cache


def exact(q, cache, n, scale):
    """Attention of the last q.shape[0] of n tokens, and sum w |v|, in 64 bits."""
    k, v = (x[:, 0].double() for x in qsa.kv_load(i32([0, n]), i32([0]), n, cache))
    s = torch.einsum("rhd,td->rht", q.double(), k) * scale
    p = torch.arange(n - q.shape[0], n, device="cuda")[:, None, None]
    s = s.masked_fill(torch.arange(n, device="cuda") > p, -float("inf"))
    w = torch.softmax(s, -1)
    return w @ v, w @ v.abs()


def attend(q, cache, n, scale):
    out = qsa.chunk_attention(q, i32([0, q.shape[0]]), i32([n - q.shape[0]]), cache, scale=scale).double()
    st = qsa.get_device_status()
    assert st == qsa.QSA_OK, qsa.status_string(st)
    return out


ROWS = pytest.mark.parametrize("rows", [1, 70])              # few rows, and units of 256 pairs
QUANT = pytest.mark.parametrize("quantised", [False, True])
DIM = pytest.mark.parametrize("D", [128, 256])


@ROWS
@QUANT
@DIM
def test_scores_past_24_bits(D, quantised, rows):
    """Scores of 5 * 2^23 and 5 * 2^24 (FP32 holds both; their products with log2 e only
    to 4 or 8): equal ones weigh the same, the smaller ones, 2^22 or more below,
    nothing.  Every product and sum of the scores is exact, the weights are equal powers
    of two, so only the value sums and the output are rounded."""
    n = 700
    g = torch.Generator(device="cuda").manual_seed(71)
    k = torch.full((n, 1, D), 4096.0, dtype=torch.float16, device="cuda")
    k[::3] = 3584.0
    v = torch.randn(n, 1, D, generator=g, device="cuda").half()
    cache = filled(k, v, quantised)
    q = torch.full((rows, 6, D), 80.0, dtype=torch.float16, device="cuda")
    out = attend(q, cache, n, 1.0)
    want, mag = exact(q, cache, n, 1.0)
    assert torch.all((out - want).abs() <= 2.0 ** -11 * want.abs() + n * 2.0 ** -24 * mag + 2.0 ** -25)


@ROWS
@QUANT
@DIM
def test_maximum_that_grows_far_from_zero(D, quantised, rows):
    """4,000 scores of 2^22, then ten of 2^22 + 6: e^6 is past 2^8, so the sums so far
    are scaled down, and the two kinds weigh about the same.  Scores are exact, and so
    are their differences; a weight is off by its FP16 rounding, 2^-11, and the
    exponential's, 2^-20 at most."""
    n = 4010
    g = torch.Generator(device="cuda").manual_seed(72)
    k = torch.zeros(n, 1, D, dtype=torch.float16, device="cuda")
    k[:, :, :64] = 256.0
    k[4000:, :, 100] = 6.0
    v = torch.randn(n, 1, D, generator=g, device="cuda").half()
    v[4000:] += 1.0
    cache = filled(k, v, quantised)
    q = torch.zeros(rows, 4, D, dtype=torch.float16, device="cuda")
    q[:, :, :64] = 256.0
    q[:, :, 100] = 1.0
    out = attend(q, cache, n, 1.0)
    want, mag = exact(q, cache, n, 1.0)
    tol = 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -18 + n * 2.0 ** -24) * mag + 2.0 ** -25
    off = (out - want).abs()
    assert torch.all(off <= tol), float((off / tol).max())


@ROWS
@DIM
def test_values_of_the_largest_size_stay_finite(D, rows):
    """All values 65,504 or its negative: so is every output.  Fifteen of sixteen
    weights are 2^-1 (1 + 0.51 * 2^-10), which FP16 rounds up by 2^-11, past what
    65,504 leaves to the border of infinity."""
    n = 2000
    k = torch.zeros(n, 1, D, dtype=torch.float16, device="cuda")
    k[:, :, 0] = -1.0
    k[::16, :, 0] = 0.0
    v = torch.full((n, 1, D), 65504.0, dtype=torch.float16, device="cuda")
    v[:, :, ::2] = -65504.0
    cache = filled(k, v, False)
    q = torch.zeros(rows, 4, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    scale = -float(np.log(0.5 * (1 + 0.51 * 2.0 ** -10)))
    out = attend(q, cache, n, scale)
    assert torch.equal(out, v[:1, :].double().expand(rows, 4, D))


@pytest.mark.parametrize("lens", [[(1, 120000)], [(70, 120000)], [(600, 9000), (1, 5000), (40, 41)], [(1, 30011), (3, 20000), (2, 7)]])
@QUANT
@DIM
def test_long_contexts_lose_no_small_weights(D, quantised, lens):
    """Unit-variance inputs.  An output is off by its rounding (2^-11), the weights'
    (2^-11 of sum w |v|, and 2^-32 of the largest weight where FP16 is subnormal, times
    the largest |v|), and the FP32 scores' (head_dim * 2^-24 * scale * sum |q k| <
    2^-12 of each weight, twice with the normalisation)."""
    g = torch.Generator(device="cuda").manual_seed(73)
    hkv, group, page = 2, 5, 64
    need = [-(-c // page) for _, c in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    perm, at = torch.randperm(sum(need), generator=torch.Generator().manual_seed(74)).to(torch.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    cache = qsa.KVCache.empty(sum(need), page, hkv, D, table.cuda(), quantised=quantised)
    T, C = sum(n for n, _ in lens), sum(c for _, c in lens)
    kv = torch.randn(C, 2 * hkv, D, generator=g, device="cuda", dtype=torch.float16)
    starts = i32(np.concatenate([[0], np.cumsum([c for _, c in lens])]).tolist())
    zero = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    qsa.kv_store(kv[:, :hkv], kv[:, hkv:], starts, zero, cache)
    k, v = qsa.kv_load(starts, zero, C, cache)
    q = torch.randn(T, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
    out = qsa.chunk_attention(q, i32(np.concatenate([[0], np.cumsum([n for n, _ in lens])]).tolist()),
                              i32([c - n for n, c in lens]), cache).double()
    st = qsa.get_device_status()
    assert st == qsa.QSA_OK, qsa.status_string(st)
    want, mag = reference64(q, k, v, lens)
    row = 0
    for n, c in lens:
        r = slice(row, row + n)
        tol = 2.0 ** -11 * want[r].abs() + 2.0 ** -10 * mag[r] + c * 2.0 ** -32 * 6.0 + 2.0 ** -25
        off = (out[r] - want[r]).abs()
        assert torch.all(off <= tol), (n, c, float((off / tol).max()))
        row += n
