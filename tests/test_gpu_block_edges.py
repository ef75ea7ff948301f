"""GPU: block_attention where it could go wrong: nothing to attend, outputs aligned
to 16 bytes, the longest block tables, offsets past 32 bits, rows that two requests
claim, waits that run out, other streams."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from kv_util import Batch
from test_gpu_block_attention import attend, check, ok, select
from test_gpu_kv_cache import device_cache, on_gpu

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens", [[(1, 300), (1, 5)], [(90, 300)]], ids=["step", "chunk"])
def test_nothing_to_attend_or_to_do(lens):
    b = Batch(61, lens, hkv=2, group=2, head_dim=128, page=16, quantised=False)
    caches = b.stored()
    out = attend(b, caches, np.zeros((b.T, 2, 0), np.int32))           # no blocks at all: zeros
    ok()
    n = int(b.seq_start[-1])
    assert not out[:n].any() and torch.all(out[n:] == 7.0)
    cache = device_cache(b, caches)
    q, _, _, ss, ps = on_gpu(b)
    sel = torch.zeros(b.T, 2, 1, dtype=torch.int32, device="cuda")
    out.fill_(7.0)
    qsa.block_attention(q, sel, i32([0]), i32([]), cache, out=out)     # no requests
    qsa.block_attention(q, sel, i32([0, 0, 0][:len(lens) + 1]), ps[:len(lens)], cache, out=out)   # empty ones
    qsa.block_attention(q[:0], sel[:0], ss, ps, cache, out=out[:0])    # no rows
    ok()
    assert torch.all(out == 7.0)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 700)], [(150, 400), (33, 33)]], ids=["step", "chunk"])
def test_output_aligned_to_16_bytes_only(lens, quantised):
    b = Batch(62, lens, hkv=2, group=3, head_dim=128, page=32, quantised=quantised)
    caches = b.stored()
    sel = select(b, 2, 63)
    q, _, _, ss, ps = on_gpu(b)
    flat = torch.full((b.T * b.hq * b.D + 8,), 7.0, dtype=torch.float16, device="cuda")
    out = flat[8:].view(b.T, b.hq, b.D)
    assert out.data_ptr() % 32 == 16
    qsa.block_attention(q, torch.from_numpy(sel).cuda(), ss, ps, device_cache(b, caches), recent=1, out=out)
    ok()
    check(b, out, caches, sel, 1)


def spread(cache, toks):
    """Keys and values [len(toks), hkv, D] of a request's tokens as float64."""
    P = cache.k.shape[1]
    page, slot = cache.block_table[0, toks // P].long(), toks % P
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if s is None:
            out.append(x[page, slot].double())
        else:
            y = x.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float().double()
            out.append(y * torch.pow(2.0, s[page, slot].double() - 127)[..., None])
    return out


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("D,page,big", [(128, 256, False), (256, 8, False), (256, 256, True)])
def test_far_positions_and_offsets_past_32_bits(D, page, big, rows, quantised):
    """The last tokens of a context of 2^25 whose table names the same pages over and
    over (a bitmap of 2^18 blocks), or a cache of more than 2^32 elements a tensor."""
    hkv, group, N = (8, 2, 1 << 14) if big else (2, 2, 1 << 25)
    pages = (1 << 32) // (page * hkv * D) + 40 if big else 40
    g = torch.Generator(device="cuda").manual_seed(5)
    some = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda")     # (of the big one, the last)
    table = some[torch.arange(N // page, device="cuda") % 37][None].contiguous()
    cache = qsa.KVCache.empty(pages, page, hkv, D, table, quantised=quantised)
    fill = torch.randn(40 * page, 2, hkv, D, generator=g, device="cuda", dtype=torch.float16)
    t40 = qsa.KVCache(cache.k, cache.v, some[None].contiguous(), cache.k_scale, cache.v_scale)
    qsa.kv_store(fill[:, 0], fill[:, 1], i32([0, 40 * page]), i32([0]), t40)
    q = torch.randn(rows, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
    last = N // 128 - 1
    sel = torch.randint(0, last, (rows, hkv, 5), generator=g, device="cuda", dtype=torch.int32)
    sel[:, :, 0], sel[:, :, 1] = last - 1, -1
    out = qsa.block_attention(q, sel, i32([0, rows]), i32([N - rows]), cache, recent=1)
    ok()
    for r in range(0, rows, 23):
        p = N - rows + r
        for h in range(hkv):
            blocks = sorted({c for c in sel[r, h].tolist() if c >= 0} | {p // 128})
            toks = torch.cat([torch.arange(128 * c, min(128 * c + 128, p + 1), device="cuda") for c in blocks])
            k, v = spread(cache, toks)
            for e in range(group):
                w = torch.softmax(q[r, h * group + e].double() @ k[:, h].T * D ** -0.5, -1)
                want, mag = w @ v[:, h], w @ v[:, h].abs()
                off = (out[r, h * group + e].double() - want).abs()
                assert torch.all(off <= 2.0 ** -11 * want.abs() + 2.0 ** -10 * mag + len(toks) * 2.0 ** -25 * 6 + 2.0 ** -25)


def test_rows_that_two_requests_claim_harm_no_other():
    """Starts that fall so that two requests overlap: any result for these two, the
    third's is right, and the call ends like any other."""
    b = Batch(64, [(40, 300), (30, 400), (60, 200)], hkv=2, group=4, head_dim=128, page=32, quantised=False)
    caches = b.stored()
    sel = select(b, 3, 65)
    table = np.concatenate([b.table[:1], b.table[:1], b.table[1:2], b.table[2:]])
    q, _, _, _, _ = on_gpu(b)
    out = torch.full((b.T, b.hq, b.D), 7.0, dtype=torch.float16, device="cuda")
    # rows 0 .. 39, then from 40 back to 20, then 20 .. 69 over the first's, then 70 ..
    ps = i32([int(b.pos_start[0]), 0, 150, int(b.pos_start[2])])
    for _ in range(3):
        qsa.block_attention(q, torch.from_numpy(sel).cuda(), i32([0, 40, 20, 70, 130]), ps, device_cache(b, caches, table), out=out)
        assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    from oracle import block_attention as O
    from kv_util import tolerance
    k, v, ks, vs = caches
    want, mag = O.attention(b.q, sel, b.seq_start, b.pos_start, b.table, k, v)
    s = slice(70, 130)
    assert np.all(np.abs(out.cpu().numpy()[s].astype(float) - want[s]) <= tolerance(want[s], mag[s], b.lens, 6.0))
    assert torch.all(out[130:] == 7.0)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("reqs,new,D,k", [(2, 1, 128, 30), (200, 1, 256, 30), (40, 2, 128, 30), (3, 400, 128, 30),
                                          (3, 400, 256, 30), (1, 6800, 128, 1024), (1, 6800, 256, 1024)])
def test_waits_that_run_out(reqs, new, D, k, quantised):
    """A limit of a nanosecond ends a call with long waits (a pair's helpers wait for the
    end of a unit of 2,000 tiles), is reported and harms nothing after it; one of a
    millisecond, far past any step, ends none."""
    g = torch.Generator(device="cuda").manual_seed(7)
    N, P, hkv, group = 1 << (15 if k < 1000 else 18), 64, 2, 4
    table = torch.randperm(N // P, generator=g, device="cuda").to(torch.int32)[None].repeat(reqs, 1)
    cache = qsa.KVCache.empty(N // P, P, hkv, D, table, quantised=quantised)
    kv = torch.randn(N, 2, hkv, D, generator=g, device="cuda", dtype=torch.float16)
    qsa.kv_store(kv[:, 0], kv[:, 1], i32([0, N]), i32([0]), cache)
    rows = reqs * new
    q = torch.randn(rows + 3, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
    sel = torch.randint(0, (N - new) // 128 - 4, (rows + 3, hkv, k), generator=g, device="cuda", dtype=torch.int32)
    ss, ps = torch.arange(reqs + 1, dtype=torch.int32, device="cuda") * new, i32([N - new] * reqs)

    def run(limit_ns):
        out = torch.full_like(q, 7.0)
        qsa.set_config(qsa.QSA_CFG_WAIT_LIMIT_NS, limit_ns)
        try:
            qsa.block_attention(q, sel, ss, ps, cache, recent=1, out=out)
        finally:
            qsa.set_config(qsa.QSA_CFG_WAIT_LIMIT_NS, 2_000_000_000)
        status = qsa.get_device_status()
        assert torch.all(out[rows:] == 7.0)
        return out, status

    first, status = run(2_000_000_000)
    assert status == qsa.QSA_OK
    for _ in range(2):
        # (a wait looks at the clock every 256 tries: a call whose waits are all shorter succeeds)
        again, status = run(1)
        long = k > 1000 and not quantised                     # (from codes, no warp waits for a unit's end)
        assert status == qsa.QSA_ERR_TIMEOUT or not long and status == qsa.QSA_OK and torch.equal(again, first)
        again, status = run(2_000_000_000)
        assert status == qsa.QSA_OK and torch.equal(again, first)
    again, status = run(1_000_000)
    assert status == qsa.QSA_OK and torch.equal(again, first)


@pytest.mark.parametrize("lens", [[(1, 700)] * 3, [(90, 700), (60, 300)]], ids=["step", "chunk"])
def test_outputs_made_for_another_stream(lens):
    """Outputs and workspace that the call makes itself, on a stream that is not the
    current one, stay its own until it is done."""
    b = Batch(66, lens, hkv=2, group=4, head_dim=128, page=32, quantised=False)
    caches = b.stored()
    sel = select(b, 3, 67)
    dsel = torch.from_numpy(sel).cuda()
    cache = device_cache(b, caches)
    q, _, _, ss, ps = on_gpu(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(30):
        outs.append(qsa.block_attention(q, dsel, ss, ps, cache, recent=1, stream=side))
        torch.full((1 << 20,), 1e4, device="cuda")          # would land in a workspace given back too early
    side.synchronize()
    torch.cuda.synchronize()
    ok()
    n = int(b.seq_start[-1])
    for out in outs:
        assert torch.equal(out[:n], outs[0][:n])
    outs[0][n:] = 7.0
    check(b, outs[0], caches, sel, 1)


def test_launch_counts():
    b = Batch(68, [(1, 300)], hkv=1, group=4, head_dim=128, page=32, quantised=False, pad_rows=0)
    cache = device_cache(b, b.stored())
    q, _, _, ss, ps = on_gpu(b)
    sel = torch.zeros(b.T, 1, 40, dtype=torch.int32, device="cuda")
    for k, want in ((3, 1), (40, 3)):                        # straight from the selections; lists, attention, join
        qsa.block_attention(q, sel[:, :, :k].contiguous(), ss[:2], ps, cache)
        assert qsa.last_launch_count() == want
    ok()


def test_a_workspace_one_byte_too_small_is_refused():
    lib = qsa.load()
    b = Batch(69, [(40, 300)], hkv=2, group=4, head_dim=128, page=32, quantised=False)
    cache = device_cache(b, b.stored())
    q, _, _, ss, ps = on_gpu(b)
    sel = torch.zeros(b.T, 2, 3, dtype=torch.int32, device="cuda")
    n = qsa.block_attention_workspace_bytes(b.T, b.hq, 2, 128, 3, 1, cache.c.max_pages * 32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty(b.T, b.hq, 128, dtype=torch.float16, device="cuda")
    for size, want in ((n - 1, qsa.QSA_ERR_WORKSPACE), (n, qsa.QSA_OK)):
        st = lib.qsa_block_attention(q.data_ptr(), q.stride(0), b.T, b.hq, 1, ss.data_ptr(), ps.data_ptr(), cache.ref,
                                     sel.data_ptr(), 3, 1, ctypes.c_float(0.1), out.data_ptr(), ws.data_ptr(), size, None)
        assert st == want
    ok()
