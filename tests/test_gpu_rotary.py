"""GPU: rotary tables and rotations against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from oracle import rotary as O

pytestmark = pytest.mark.gpu

SCALINGS = [None, ("linear", 4.0, {}), ("base", 4.0, {}),
            ("parts", 8.5, dict(original=2048.0, fast=32.0, slow=1.0, amplitude=1.2))]


def freqs(n, theta, scaling):
    if scaling is None:
        return O.frequencies(n, theta), 1.0, None
    kind, factor, kw = scaling
    f = O.frequencies(n, theta, kind, factor, kw.get("original", 0.0), kw.get("fast", 32.0), kw.get("slow", 1.0))
    return f, kw.get("amplitude", 1.0), qsa.RopeScaling(kind, factor, **kw)


def ok():
    st = qsa.get_device_status()
    assert st == qsa.QSA_OK, qsa.status_string(st)


@pytest.mark.parametrize("scaling", SCALINGS, ids=["none", "linear", "base", "parts"])
@pytest.mark.parametrize("n_pos,dim,theta", [(1, 16, 1e4), (777, 64, 1e4), (200001, 128, 1e6), (300, 256, 10.0)])
def test_table(n_pos, dim, theta, scaling):
    f, amp, sc = freqs(dim, theta, scaling)
    got = qsa.rotary_table(n_pos, dim, theta, sc)
    ok()
    p = np.unique(np.concatenate([np.arange(min(n_pos, 50)), np.linspace(0, n_pos - 1, 40).astype(int)]))
    angle = p[:, None] * f
    want = amp * np.concatenate([np.cos(angle), np.sin(angle)], 1)
    # FP32's rounding (2^-24 of the value, 2^-150 at least), and the angle's error in FP64:
    # the frequency is off by a few units of 2^-53, so the angle by 2^-50 of itself
    tol = 2.0 ** -24 * np.abs(want) + amp * 2.0 ** -50 * (1 + np.abs(np.concatenate([angle, angle], 1))) + 2.0 ** -140
    off = np.abs(got.cpu().numpy()[p].astype(np.float64) - want)
    assert np.all(off <= tol), np.max(off / tol)


def batch(lens, hq, hk, D, seed, pad=3):
    rng = np.random.default_rng(seed)
    ss = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    ps = np.array([c - n for n, c in lens], np.int32)
    T = int(ss[-1]) + pad
    fused = rng.standard_normal((T, hq + hk + 1, D)).astype(np.float16)
    pos = np.zeros(T)
    for b, (n, c) in enumerate(lens):
        pos[ss[b]:ss[b + 1]] = np.arange(c - n, c)
    return fused, ss, ps, pos


def tolerance(x, want, amp):
    """One rounding to FP16 (2^-11 of the value, half its finest step at least), and of
    the FP32 sum: the table's rounding, two products and a sum, each within 2^-24 of
    the pair's length times the amplitude."""
    size = amp * np.sqrt(2.0) * np.abs(x.astype(np.float64)).max()
    return 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 4 * 2.0 ** -24 * size


CASES = [  # lens, hq, hk, D, first, rope
    ([(1, 1), (1, 500), (1, 30)], 24, 2, 256, 0, 64), ([(37, 300)], 5, 1, 128, 0, 128), ([(3, 9), (0, 4), (70, 90)], 1, 1, 64, 16, 48),
    ([(1, 5)], 32, 8, 128, 64, 64), ([(130, 130), (9, 1000)], 3, 0, 192, 8, 176), ([(20, 999)], 7, 3, 512, 248, 256),
    ([(1, 2)] * 700, 2, 1, 16, 0, 16), ([(2, 2)], 300, 20, 32, 0, 32)]


@pytest.mark.parametrize("scaling", [SCALINGS[0], SCALINGS[3]], ids=["none", "parts"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,hq,hk,D,first,rope", CASES)
def test_rotation(lens, hq, hk, D, first, rope, in_place, interleaved, scaling):
    f, amp, sc = freqs(rope, 1e4, scaling)
    fused, ss, ps, pos = batch(lens, hq, hk, D, 61)
    x = torch.from_numpy(fused).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    tab = qsa.rotary_table(max(c for _, c in lens), rope, 1e4, sc)
    args = (q, k, torch.from_numpy(ss).cuda(), torch.from_numpy(ps).cuda(), tab)
    n, before = int(ss[-1]), x.clone()
    if in_place:
        oq, ok_ = qsa.rotary(*args, first=first, interleaved=interleaved, out_q=q, out_k=k)
        assert oq is q and ok_ is k
        assert torch.equal(x[n:], before[n:]) and torch.equal(x[:, hq + hk:], before[:, hq + hk:])
    else:
        out = torch.full_like(x, 7.0)                       # rows of a wider array
        outs = dict(out_q=out[:, 1:hq + 1], out_k=out[:, hq + 1:] if hk else None)
        oq, ok_ = qsa.rotary(*args, first=first, interleaved=interleaved, **outs)
        assert torch.equal(x, before) and torch.all(out[n:] == 7.0) and torch.all(out[:, 0] == 7.0)
    ok()
    for got, src in [(oq, fused[:, :hq])] + ([(ok_, fused[:, hq:hq + hk])] if hk else []):
        want = O.rotate(src, pos, f, first, interleaved, amp)[:n]
        got = got.cpu().numpy()[:n].astype(np.float64)
        off = np.abs(got - want)
        assert np.all(off <= tolerance(src, want, amp))
        rest = [d for d in range(D) if not first <= d < first + rope]
        np.testing.assert_array_equal(got[..., rest], src[:n].astype(np.float64)[..., rest])


def test_outputs_are_made_and_one_of_two_in_place():
    fused, ss, ps, pos = batch([(50, 80)], 4, 2, 64, 62, pad=0)
    x = torch.from_numpy(fused).cuda()
    q, k = x[:, :4], x[:, 4:6].contiguous()
    tab = qsa.rotary_table(80, 32)
    args = (torch.from_numpy(ss).cuda(), torch.from_numpy(ps).cuda(), tab)
    f = O.frequencies(32, 1e4)
    oq, ok_ = qsa.rotary(q, k, *args)
    assert oq.is_contiguous() and ok_.is_contiguous()
    o2, k2 = qsa.rotary(q, k, *args, out_k=k)
    ok()
    assert k2 is k and torch.equal(o2, oq) and torch.equal(k2, ok_)
    want = O.rotate(fused[:, :4], pos, f, 0, False)
    assert np.all(np.abs(oq.cpu().numpy().astype(float) - want) <= tolerance(fused, want, 1.0))


def test_special_values():
    """Infinities and NaN stay in their pair; results past FP16 become infinite."""
    x = np.zeros((2, 3, 16), np.float16)
    x[:, 0, 0], x[:, 1, 1], x[:, 2, 2], x[:, 2, 10] = np.inf, np.nan, 65504, -65504
    q = torch.from_numpy(x).cuda()
    tab = qsa.rotary_table(2, 16)
    one = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    got, _ = qsa.rotary(q, None, one(0, 2), one(0), tab)
    ok()
    got = got.cpu().numpy()
    c, s = np.cos(1 * 10.0 ** -1), np.sin(1 * 10.0 ** -1)               # pair 2 of 8: 10^4 to the -2 * 2 / 16
    np.testing.assert_allclose(got[1, 2, [2, 10]].astype(float), [np.inf, 65504 * (s - c)], rtol=2.0 ** -11)
    assert np.isinf(got[1, 0, 0]) and np.isinf(got[1, 0, 8]) and np.isnan(got[:, 1, 1]).all()
    other = np.ones(16, bool)
    other[[0, 8, 1, 9, 2, 10]] = False
    assert not got[:, :, other].any()


def test_bad_requests():
    fused, ss, ps, pos = batch([(4, 9), (3, 50), (2, 20), (5, 30)], 2, 1, 64, 63)
    x = torch.from_numpy(fused).cuda()
    tab = qsa.rotary_table(30, 64)                          # the second request lies past the table
    ps[2] = -1
    out = torch.full((x.shape[0], 2, 64), 7.0, dtype=torch.float16, device="cuda")
    qsa.rotary(x[:, :2], None, torch.from_numpy(ss).cuda(), torch.from_numpy(ps).cuda(), tab, out_q=out)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    want = O.rotate(fused[:, :2], pos, O.frequencies(64, 1e4), 0, False)
    got = out.cpu().numpy().astype(float)
    for r in range(4):
        s = slice(ss[r], ss[r + 1])
        if r in (1, 2):
            assert np.all(got[s] == 7.0)
        else:
            assert np.all(np.abs(got[s] - want[s]) <= tolerance(fused, want[s], 1.0))
    assert np.all(got[ss[-1]:] == 7.0)
    # starts that fall: the requests that are well formed are served
    out.fill_(7.0)
    one = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    qsa.rotary(x[:, :2], None, one(7, 14, 0, 7), one(3, 0, 1), tab, out_q=out)
    assert qsa.get_device_status() == qsa.QSA_ERR_INVALID_ARG
    pos = np.concatenate([1 + np.arange(7), 3 + np.arange(7), np.zeros(3)])
    want = O.rotate(fused[:, :2], pos, O.frequencies(64, 1e4), 0, False)[:14]
    got = out.cpu().numpy().astype(float)
    assert np.all(np.abs(got[:14] - want) <= tolerance(fused, want, 1.0)) and np.all(got[14:] == 7.0)


def test_graph_and_stream():
    fused, ss, ps, pos = batch([(1, 40)] * 5, 4, 1, 128, 64, pad=0)
    x = torch.from_numpy(fused).cuda()
    tab = qsa.rotary_table(100, 64)
    sst, pst = torch.from_numpy(ss).cuda(), torch.from_numpy(ps).cuda()
    out = torch.empty(5, 4, 128, dtype=torch.float16, device="cuda")
    qsa.rotary(x[:, :4], None, sst, pst, tab, out_q=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.rotary(x[:, :4], None, sst, pst, tab, out_q=out)
    pst.add_(7)
    g.replay()
    side = torch.cuda.Stream()
    got, gk = qsa.rotary(x[:, :4], x[:, 4:5], sst, pst, tab, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    ok()
    want = O.rotate(fused[:, :4], pos + 7, O.frequencies(64, 1e4), 0, False)
    for y in (out, got):
        assert np.all(np.abs(y.cpu().numpy().astype(float) - want) <= tolerance(fused, want, 1.0))


def test_refusals_in_python():
    x = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    tab = qsa.rotary_table(8, 32)
    call = lambda **kw: qsa.rotary(**{**dict(q=x, k=x, seq_start=i, pos_start=i[:2], table=tab), **kw})  # noqa: E731
    for kw, err in [(dict(q=x.float()), TypeError), (dict(k=x[:2]), ValueError), (dict(k=x.cpu()), ValueError),
                    (dict(table=tab.half()), ValueError), (dict(table=tab[:, :16]), ValueError), (dict(pos_start=i), ValueError),
                    (dict(out_q=x[:, :1].contiguous()), ValueError), (dict(k=None, out_k=x), ValueError),
                    (dict(q=x.transpose(0, 1)), ValueError), (dict(first=40), qsa.QSAError), (dict(first=4), qsa.QSAError)]:
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(qsa.QSAError):
        qsa.rotary_table(8, 24)
