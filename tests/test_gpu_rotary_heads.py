"""GPU: rotary where a thread goes through several batches of heads, in both layouts, in
place and not."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from oracle import rotary as O
from test_gpu_rotary import batch, ok, tolerance

pytestmark = pytest.mark.gpu

# lens, hq, hk, D, first, rope: prompts (ten heads to a thread, in batches of four), the
# same with a number of heads that is no multiple of anything; few rows of many heads; the
# widest heads, whose pieces leave room for eight threads to a row
CASES = [([(3000, 3000), (1, 50), (2200, 4000)], 32, 8, 128, 0, 128), ([(5200, 5200)], 31, 6, 128, 16, 96),
         ([(2, 9), (1, 70)], 300, 21, 64, 0, 64), ([(3, 9)], 37, 0, 512, 0, 64), ([(2, 30), (9, 9)], 29, 10, 512, 248, 256),
         ([(1, 3)], 600, 3, 512, 8, 256)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,hq,hk,D,first,rope", CASES)
def test_many_heads(lens, hq, hk, D, first, rope, in_place, interleaved):
    f = O.frequencies(rope, 1e4)
    fused, ss, ps, pos = batch(lens, hq, hk, D, 65)
    x = torch.from_numpy(fused).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    tab = qsa.rotary_table(max(c for _, c in lens), rope)
    args = (q, k, torch.from_numpy(ss).cuda(), torch.from_numpy(ps).cuda(), tab)
    n, before = int(ss[-1]), x.clone()
    if in_place:
        got = x
        qsa.rotary(*args, first=first, interleaved=interleaved, out_q=q, out_k=k)
    else:
        got = torch.full_like(x, 7.0)
        qsa.rotary(*args, first=first, interleaved=interleaved, out_q=got[:, :hq], out_k=got[:, hq:hq + hk] if hk else None)
        assert torch.equal(x, before)
        before = torch.full_like(x, 7.0)
    ok()
    assert torch.equal(got[n:], before[n:]) and torch.equal(got[:, hq + hk:], before[:, hq + hk:])
    rows = np.unique(np.concatenate([np.arange(0, n, 1 + n // 300), [n - 1]]))
    want = O.rotate(fused[rows, :hq + hk], pos[rows], f, first, interleaved)
    here = got[torch.from_numpy(rows).cuda(), :hq + hk].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(here - want) <= tolerance(fused, want, 1.0))
    # every row against the 32-bit formula on the device, within twice that
    c, s = (t.float()[:, None] for t in tab[torch.from_numpy(pos[:n]).long().cuda()].split(rope // 2, 1))
    src = torch.from_numpy(fused[:n, :hq + hk]).cuda().float()
    turn = src[..., first:first + rope].unflatten(-1, (-1, 2) if interleaved else (2, -1))
    a, b = turn.unbind(-1 if interleaved else -2)
    src[..., first:first + rope] = torch.stack([a * c - b * s, b * c + a * s], -1 if interleaved else -2).flatten(-2)
    off = (got[:n, :hq + hk].float() - src).abs()
    size = np.sqrt(2.0) * np.abs(fused.astype(np.float64)).max()
    assert torch.all(off <= 2.0 ** -11 * src.abs() * (1 + 2.0 ** -10) + 2.0 ** -25 + 8 * 2.0 ** -24 * size)
