"""GPU: block_attention and its neighbours on paths between the ordinary ones: kernels
that may not start early, captured decode steps with many more rows than tokens, memory
that a call makes itself while its stream is behind."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import Batch
from test_gpu_block_attention import attend, check, ok, select
from test_gpu_kv_cache import device_cache, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("lens,group,D", [([(3, 900), (2, 700), (1, 40)], 4, 128), ([(2, 900), (2, 1700)], 8, 256),
                                          ([(150, 1400), (60, 300)], 12, 128), ([(150, 1400), (60, 300)], 12, 256)],
                         ids=["few-128", "few-256", "many-128", "many-256"])
def test_without_early_starts(lens, group, D, quantised):
    """QSA_CFG_OVERLAP 0: lists, attention and join one after the other, the same bits."""
    b = Batch(81, lens, hkv=2, group=group, head_dim=D, page=32, quantised=quantised)
    caches = b.stored()
    sel = select(b, 4, 82)
    first = attend(b, caches, sel, 1)
    assert qsa.last_launch_count() == 3
    qsa.set_config(qsa.QSA_CFG_OVERLAP, 0)
    try:
        again = [attend(b, caches, sel, 1) for _ in range(3)]
        assert qsa.last_launch_count() == 3
    finally:
        qsa.set_config(qsa.QSA_CFG_OVERLAP, 1)
    ok()
    check(b, first, caches, sel, 1)
    for out in again:
        assert torch.equal(out, first)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("D,group", [(128, 12), (256, 1), (128, 20)])
def test_captured_decode_step_of_many_more_rows_than_tokens(D, group, quantised):
    """A graph for padded rows (which choose the kernel for many) against the same tokens
    by themselves (the kernel for few), both held to the oracle."""
    lens = [(1, 700), (1, 129), (1, 1500)]
    b = Batch(83, lens, hkv=2, group=group, head_dim=D, page=64, quantised=quantised, pad_rows=557)
    caches = b.stored()
    sel = select(b, 5, 84)
    q, _, _, ss, ps = on_gpu(b)
    dsel, cache = torch.from_numpy(sel).cuda(), device_cache(b, caches)
    out = torch.empty(b.T, b.hq, D, dtype=torch.float16, device="cuda")
    ws = qsa.alloc_block_attention_workspace(cache, b.T, b.hq, 5, 1)
    qsa.block_attention(q, dsel, ss, ps, cache, recent=1, out=out, ws=ws)
    assert qsa.last_launch_count() == 3
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.block_attention(q, dsel, ss, ps, cache, recent=1, out=out, ws=ws)
    start = b.pos_start.copy()
    for back in (0, 60, 128):                                # (positions of the replay, not of the capture)
        b.pos_start = start - back
        b.lens = [(n, c - back) for n, c in lens]
        ps.copy_(torch.from_numpy(b.pos_start))
        near = np.minimum(sel[:3], (b.pos_start // 128)[:, None, None])
        dsel[:3] = torch.from_numpy(near).cuda()
        out.fill_(7.0)
        g.replay()
        alone = qsa.block_attention(q[:3], dsel[:3], ss, ps, cache, recent=1)
        assert qsa.last_launch_count() == (1 if group <= 16 else 3)
        ok()
        here = np.concatenate([near, sel[3:]])
        check(b, out, caches, here, 1)
        out[:3] = alone
        check(b, out, caches, here, 1)


def overlaps(t, start, size):
    return t.data_ptr() < start + size and start < t.data_ptr() + t.numel() * t.element_size()


@pytest.mark.parametrize("lens,group,k", [([(1, 700)] * 3, 4, 40), ([(90, 700), (60, 300)], 4, 3), ([(1, 700)] * 3, 4, 3)],
                         ids=["lists-few", "lists-many", "straight"])
def test_memory_made_for_a_stream_that_is_behind(lens, group, k, monkeypatch):
    """Workspace and output that a call makes itself, for a stream that has not come to
    it yet, are handed out to nobody else, although the caller has dropped them."""
    b = Batch(85, lens, hkv=2, group=group, head_dim=128, page=32, quantised=False, pad_rows=0)
    caches = b.stored()
    sel = select(b, k, 86)
    dsel, cache = torch.from_numpy(sel).cuda(), device_cache(b, caches)
    q, kn, _, ss, ps = on_gpu(b)
    tab = qsa.rotary_table(2000, 64)
    made = []
    plain = qsa.alloc_block_attention_workspace

    def noted(*a):
        ws = plain(*a)
        made.append((ws.data_ptr(), ws.numel()))
        return ws

    monkeypatch.setattr(qsa, "alloc_block_attention_workspace", noted)
    qsa.block_attention(q, dsel, ss, ps, cache, recent=1)     # (loads the kernels)
    assert qsa.last_launch_count() == (1 if k < 32 and lens[0][0] == 1 else 3)
    qsa.rotary(q, kn, ss, ps, tab)
    torch.cuda.synchronize()
    made.clear()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                       # some 0.1 s
    out = qsa.block_attention(q, dsel, ss, ps, cache, recent=1, stream=side)
    rq, rk = qsa.rotary(q, kn, ss, ps, tab, stream=side)
    copy = torch.empty_like(out)
    with torch.cuda.stream(side):
        copy.copy_(out)
    copy.record_stream(side)
    made += [(x.data_ptr(), x.numel() * 2) for x in (out, rq, rk)]
    assert len(made) == 4 and not side.query()
    del out, rq, rk
    fill = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _, size in made for _ in range(4)]
    assert not side.query()
    for t in fill:
        assert not any(overlaps(t, start, size) for start, size in made)
    side.synchronize()
    ok()
    check(b, copy, caches, sel, 1)


@pytest.mark.parametrize("D,hkv,group", [(128, 2, 8), (256, 2, 12)])
def test_many_rows_over_an_fp16_copy_of_an_e4m3_context(D, hkv, group):
    """Contexts read back into rows that serve as another cache's pages: the same bits."""
    P, lens = 32, [(300, 960), (270, 288), (1, 1408)]
    b = Batch(87, lens, hkv=hkv, group=group, head_dim=D, page=P, quantised=True)
    cache = device_cache(b, b.stored())
    q, _, _, ss, ps = on_gpu(b)
    dsel = torch.from_numpy(select(b, 4, 88)).cuda()
    want = qsa.block_attention(q, dsel, ss, ps, cache, recent=1)
    ends = np.cumsum([0] + [c for _, c in lens]).astype(np.int32)
    k, v = qsa.kv_load(torch.from_numpy(ends).cuda(), torch.zeros_like(ps), int(ends[-1]), cache)
    table = torch.full((3, 44), -1, dtype=torch.int32, device="cuda")
    for r, (_, c) in enumerate(lens):
        table[r, :c // P] = torch.arange(c // P, device="cuda") + int(ends[r]) // P
    half = qsa.KVCache(k.view(-1, P, hkv, D), v.view(-1, P, hkv, D), table)
    got = qsa.block_attention(q, dsel, ss, ps, half, recent=1)
    assert qsa.last_launch_count() == 3
    ok()
    n = int(b.seq_start[-1])
    assert torch.equal(got[:n], want[:n])
