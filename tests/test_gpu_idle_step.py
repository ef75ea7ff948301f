"""GPU: a padded step without rows, and padding rows whose request has given its first
page back, end without an error; a first token without a page is still reported."""
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa

pytestmark = pytest.mark.gpu

P, HKV, K, ROWS, PAGES = 128, 2, 3, 300, 6


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """A layer's step over three requests, for both row-map consumers (the scorer reads
    128-wide keys, sparse attention 256-wide heads)."""

    def __init__(self, entry):
        g = torch.Generator(device="cuda").manual_seed(3)
        h = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
        self.table = torch.full((3, 4), entry, dtype=torch.int32, device="cuda")
        self.cache = qsa.KVCache(h(PAGES, P, HKV, 128), h(PAGES, P, HKV, 128), self.table)
        self.wide = h(PAGES, P, HKV, 256), h(PAGES, P, HKV, 256)
        e = qsa.Batch.empty(3, ROWS, "cuda")
        self.lens = torch.zeros(3, dtype=torch.int32, device="cuda")
        self.batch = qsa.Batch(e.seq_start, e.pos_start, self.lens, e.row_req, e.row_token, e.row_visible, e.slot, e.state)
        self.batch.state.copy_(i32(0, PAGES, 0))
        self.free, self.new = torch.arange(PAGES, dtype=torch.int32, device="cuda"), i32(0, 0, 0)
        self.q, self.kv, self.qi, self.q2 = h(ROWS, 4, 128), h(ROWS, HKV, 128), h(ROWS, HKV, 128), h(ROWS, 4, 256)
        self.rope = qsa.rotary_table(P * 4, 64)
        self.sel, self.none = (torch.full((ROWS, n, K), -1, dtype=torch.int32, device="cuda") for n in (HKV, 1))
        self.val = torch.zeros(ROWS, HKV, K, device="cuda")
        self.out, self.wide_out = torch.full_like(self.q, 7.0), torch.zeros(ROWS, 4, 256, device="cuda")

    def tables(self):
        qsa.batch_tables(self.new, self.lens, self.free, self.batch.state[1:2], self.table, P, self.batch)

    def consumers(self):
        b = self.batch
        qsa.block_select(self.qi, self.cache.k, self.table, b.row_req, b.row_token, K, out_idx=self.sel, out_val=self.val)
        qsa.sparse_attention(self.q2, *self.wide, self.table, b.row_req, b.row_token, self.none[:, 0].contiguous(),
                             out=self.wide_out)

    def run(self):
        b = self.batch
        self.tables()
        qsa.rotary(self.q, self.kv, b.seq_start, b.pos_start, self.rope, out_q=self.q, out_k=self.kv)
        qsa.kv_store(self.kv, self.kv, b.seq_start, b.pos_start, self.cache)
        self.consumers()
        qsa.block_attention(self.q, self.sel, b.seq_start, b.pos_start, self.cache, recent=1, out=self.out)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1, 1000])
def test_steps_without_rows(entry, graph):
    """No request has a page yet (its entries hold anything); nothing new, or too much to fit."""
    s = Step(entry)
    run = s.run
    if graph:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        run = g.replay
    before = s.q.clone()
    for new in ((0, 0, 0), (ROWS + 1, 5, 5), (0, ROWS + 1, 0)):
        s.new.copy_(i32(*new))
        s.out.fill_(7.0)
        run()
        assert qsa.get_device_status() == qsa.QSA_OK, new
        assert s.batch.state[:2].tolist() == [0, PAGES] and torch.all(s.table == entry)
        assert torch.equal(s.q, before) and torch.all(s.out == 7.0)
        assert torch.all(s.sel == -1) and torch.all(torch.isneginf(s.val)) and not s.wide_out.any()
    s.new.copy_(i32(200, 0, 3))                              # then the requests begin
    run()
    assert qsa.get_device_status() == qsa.QSA_OK
    assert s.batch.state.tolist() == [203, PAGES - 3, 3] and torch.all(s.sel[:203, :, 0] >= 0)
    assert not torch.any(s.out[:203] == 7.0) and torch.all(s.out[203:] == 7.0)


def test_padding_of_a_request_that_gave_its_first_page_back():
    """A window's pages go back to the list: rows behind the batch, which name the last
    row's request and token 0, are passed over beside rows of that request."""
    s = Step(-1)
    s.new.copy_(i32(0, 300, 0))
    s.run()
    s.table[1, 0] = -1
    s.new.copy_(i32(0, 2, 0))
    s.tables()
    b = s.batch
    assert b.row_req.tolist() == [1] * ROWS and b.row_token[:3].tolist() == [300, 301, 0]
    b.row_token[:2] = 0                                      # (rows further on would score the first block, too)
    s.consumers()
    assert qsa.get_device_status() == qsa.QSA_OK
    assert torch.all(s.sel == -1) and not s.wide_out.any()
    s.table[1, 0] = 0
    want, _ = qsa.block_select(s.qi, s.cache.k, s.table, b.row_req, b.row_token, K)
    s.table[2, 0], b.row_req[2:] = -1, 2                     # rows of request 1 beside padding of request 2
    s.consumers()
    assert qsa.get_device_status() == qsa.QSA_OK
    assert torch.equal(s.sel[:2], want[:2]) and torch.all(s.sel[2:] == -1) and torch.all(want[:, :, 0] == 0)


@pytest.mark.parametrize("token", [1, 127, 300])
def test_later_tokens_without_a_page_are_reported(token):
    s = Step(-1)
    b = s.batch
    b.row_req.fill_(1), b.row_token.fill_(token)
    s.table[1, 1:] = i32(1, 2, 3)
    qsa.block_select(s.qi, s.cache.k, s.table, b.row_req, b.row_token, K)
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE
    s.table[1] = -1
    qsa.sparse_attention(s.q2, *s.wide, s.table, b.row_req, b.row_token, s.none[:, 0].contiguous())
    assert qsa.get_device_status() == (qsa.QSA_ERR_BAD_PAGE if (token + 1) % 4 else qsa.QSA_OK)
    # the store reports a first token without a page
    qsa.kv_store(s.kv, s.kv, i32(0, 1, 1, 1), i32(0, 0, 0), s.cache)
    assert qsa.get_device_status() == qsa.QSA_ERR_BAD_PAGE


def test_rows_with_a_bad_request_or_token_are_reported():
    s = Step(-1)
    b = s.batch
    for req, token in ((3, 0), (-1, 0), (0, -1)):
        b.row_req.fill_(req), b.row_token.fill_(token)
        s.consumers()
        assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
