"""GPU: chunk_attention when a wait of its pipeline runs out, and when none may.

80 units of 256 pairs over up to 800,000 tokens: a pair of SMs is at one unit for
some ten milliseconds, and its helper warps wait for the unit's end."""
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa

pytestmark = pytest.mark.gpu

TOKENS, ROWS, GROUP = 800_000, 1700, 12


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(params=[128, 256], scope="module")
def call(request):
    D, page = request.param, 64
    g = torch.Generator(device="cuda").manual_seed(81)
    table = torch.randperm(TOKENS // page, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    cache = qsa.KVCache.empty(TOKENS // page, page, 1, D, table)
    kv = torch.randn(TOKENS, 2, D, generator=g, device="cuda", dtype=torch.float16)
    qsa.kv_store(kv[:, :1], kv[:, 1:], i32([0, TOKENS]), i32([0]), cache)
    q = torch.randn(ROWS + 5, GROUP, D, generator=g, device="cuda", dtype=torch.float16)
    ss, ps = i32([0, ROWS]), i32([TOKENS - ROWS])

    def run(limit_ns):
        out = torch.full_like(q, 7.0)
        qsa.set_config(qsa.QSA_CFG_WAIT_LIMIT_NS, limit_ns)
        try:
            qsa.chunk_attention(q, ss, ps, cache, out=out)
        finally:
            qsa.set_config(qsa.QSA_CFG_WAIT_LIMIT_NS, 2_000_000_000)
        status = qsa.get_device_status()
        assert torch.all(out[ROWS:] == 7.0)
        return out, status

    return run


def test_a_wait_that_runs_out_is_reported_and_harms_nothing_after(call):
    first, status = call(2_000_000_000)
    assert status == qsa.QSA_OK
    for _ in range(3):
        assert call(1)[1] == qsa.QSA_ERR_TIMEOUT
        again, status = call(2_000_000_000)
        assert status == qsa.QSA_OK
        assert torch.equal(again, first)


def test_a_limit_of_a_step_does_not_end_a_long_unit(call):
    first, status = call(2_000_000_000)
    assert status == qsa.QSA_OK
    again, status = call(1_000_000)                          # a millisecond, for steps of two microseconds
    assert status == qsa.QSA_OK
    assert torch.equal(again, first)


@pytest.mark.parametrize("limit_ns", [2 ** 62, 2 ** 63 - 1])
def test_the_largest_limit_is_no_limit(call, limit_ns):
    first, status = call(2_000_000_000)
    assert status == qsa.QSA_OK
    again, status = call(limit_ns)
    assert status == qsa.QSA_OK
    assert torch.equal(again, first)
