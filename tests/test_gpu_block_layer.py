"""GPU: one layer's operators as a serving step runs them: tables from lengths,
rotary positions, K/V store, block selection, attention over the selected blocks."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import tolerance
from oracle import batch_tables as BT
from oracle import block_attention as BA
from oracle import block_scorer as BS
from oracle import rotary as R

pytestmark = pytest.mark.gpu

HKV, GROUP, D, P, K, ROPE = 2, 4, 128, 128, 3, 64


def ok():
    st = qsa.get_device_status()
    assert st == qsa.QSA_OK, qsa.status_string(st)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_prompts_then_decode(graph):
    """Three requests grow, chunk by chunk and token by token, in a padded batch."""
    rng = np.random.default_rng(80)
    steps = [[300, 150, 0], [200, 1, 129], [1, 1, 260], [1, 1, 1], [1, 0, 1], [2, 3, 1]]
    rows, n = 560, 3
    total = np.sum(steps, 0)
    pages, max_pages = int(sum(-(-t // P) for t in total)) + 4, 8
    free_np = rng.permutation(pages).astype(np.int32)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")
    cache = qsa.KVCache(f16(pages, P, HKV, D), f16(pages, P, HKV, D), table)
    e = qsa.Batch.empty(n, rows, "cuda")
    lens = i32(n)
    batch = qsa.Batch(e.seq_start, e.pos_start, lens, e.row_req, e.row_token, e.row_visible, e.slot, e.state)
    batch.state.copy_(torch.tensor([0, pages, 0], dtype=torch.int32))
    free, new = torch.from_numpy(free_np).cuda(), i32(n)
    hq = HKV * GROUP
    fused = f16(rows, hq + 2 * HKV, D)
    qi = f16(rows, HKV, D)                                # the scorer's queries
    rope = qsa.rotary_table(2000, ROPE)
    q, k, v = fused[:, :hq], fused[:, hq:hq + HKV], fused[:, hq + HKV:]
    sel = i32(rows, HKV, K)
    val = torch.zeros(rows, HKV, K, device="cuda")
    out = torch.full((rows, hq, D), 7.0, dtype=torch.float16, device="cuda")
    ws = qsa.alloc_block_attention_workspace(cache, rows, hq, K, 1)
    ws_sel = torch.empty(int(qsa.load().qsa_block_select_workspace_bytes(rows, HKV, max_pages, K)), dtype=torch.uint8,
                         device="cuda")

    def step():
        qsa.batch_tables(new, lens, free, batch.state[1:2], table, P, batch)
        qsa.rotary(q, k, batch.seq_start, batch.pos_start, rope, out_q=q, out_k=k)
        qsa.kv_store(k, v, batch.seq_start, batch.pos_start, cache)
        qsa.block_select(qi, cache.k, table, batch.row_req, batch.row_token, K, out_idx=sel, out_val=val, ws=ws_sel)
        qsa.block_attention(q, sel, batch.seq_start, batch.pos_start, cache, recent=1, out=out, ws=ws)

    run = step
    if graph:
        step()                                            # no tokens yet: padding names a request without pages
        assert qsa.get_device_status() in (qsa.QSA_OK, qsa.QSA_ERR_BAD_PAGE)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    lens_np, table_np, left = np.zeros(n, np.int32), np.full((n, max_pages), -1, np.int32), pages
    kc = np.zeros((pages, P, HKV, D), np.float16)
    vc = np.zeros_like(kc)
    f = R.frequencies(ROPE, 1e4)
    for s in steps:
        x = rng.standard_normal((rows, hq + 2 * HKV, D)).astype(np.float16)
        xi = rng.standard_normal((rows, HKV, D)).astype(np.float16)
        fused.copy_(torch.from_numpy(x))
        qi.copy_(torch.from_numpy(xi))
        new.copy_(torch.tensor(s, dtype=torch.int32))
        out.fill_(7.0)
        run()
        ok()
        want, _ = BT.tables(s, lens_np, rows, P, table_np, free_np, left)
        ctx, lens_np, table_np, left = lens_np, want["total_len"], want["block_table"], int(want["state"][1])
        np.testing.assert_array_equal(table.cpu().numpy(), table_np)
        np.testing.assert_array_equal(batch.slot.cpu().numpy(), want["slot"])
        T = int(want["seq_start"][-1])
        # each later stage from what the stage before it left on the device
        rot = R.rotate(x[:T, :hq + HKV], want["row_token"][:T], f, 0, False)
        got = fused.cpu().numpy()
        assert np.all(np.abs(got[:T, :hq + HKV] - rot) <= 2.0 ** -11 * np.abs(rot) + 2.0 ** -20)
        np.testing.assert_array_equal(got[T:], x[T:])
        kc.reshape(-1, HKV, D)[want["slot"][:T]] = got[:T, hq:hq + HKV]
        vc.reshape(-1, HKV, D)[want["slot"][:T]] = x[:T, hq + HKV:]
        np.testing.assert_array_equal(cache.k.cpu().numpy(), kc)
        np.testing.assert_array_equal(cache.v.cpu().numpy(), vc)
        picked = sel.cpu().numpy()
        for r in range(0, T, 7):                          # scores are FP32 sums: the picked ones' values, and none better
            b, tok = want["row_req"][r], want["row_token"][r]
            pg = table_np[b, :tok // P + 1]
            for h in range(HKV):
                sc = BS.block_scores(xi[r, h], kc[pg, :, h].reshape(-1, D), tok)
                mine = picked[r, h][picked[r, h] >= 0]
                assert len(mine) == min(K, len(sc)) and len(set(mine)) == len(mine)
                rest = np.delete(sc, mine)
                assert rest.size == 0 or sc[mine].min() >= rest.max() - 1e-3
        o, mag = BA.attention(got[:T, :hq], picked[:T], want["seq_start"], ctx, table_np, kc, vc, recent=1)
        res = out.cpu().numpy().astype(np.float64)
        tol = tolerance(o, mag, [(0, int(lens_np.max()))], 6.0)
        assert np.all(np.abs(res[:T] - o) <= tol)
        assert np.all(res[T:] == 7.0)
    assert lens_np.tolist() == total.tolist()
