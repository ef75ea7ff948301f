"""batch_tables, rotary and block_attention on a machine without a GPU: what they
refuse before any launch."""
import ctypes

import pytest
import torch

from block_sparse_attention_select_gb300 import build as qbuild
from block_sparse_attention_select_gb300 import qsa
from test_kv_host import _cache

vp = ctypes.c_void_p
BAD, UNSUP, GO = qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_UNSUPPORTED, qsa.QSA_ERR_NO_DEVICE


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def _tables(lib, batch=None, **kw):
    a = dict(new=16, ctx=16, n=2, rows=8, P=64, table=16, mp=4, free=16, cap=3, count=16)
    a.update(kw)
    arrays = dict.fromkeys(qsa.Batch._NAMES, 16)
    arrays.update(batch or {})
    c = qsa.BatchC(*arrays.values())
    return lib.qsa_batch_tables(vp(a["new"]), vp(a["ctx"]), a["n"], a["rows"], a["P"], vp(a["table"]), a["mp"],
                                vp(a["free"]), a["cap"], vp(a["count"]), ctypes.byref(c), None)


def test_tables(lib):
    for kw, want in [(dict(n=-1), BAD), (dict(rows=-1), BAD), (dict(mp=0), BAD), (dict(cap=-1), BAD),
                     (dict(new=None), BAD), (dict(ctx=None), BAD), (dict(table=None), BAD), (dict(count=None), BAD),
                     (dict(free=None), BAD), (dict(new=18), BAD), (dict(ctx=18), BAD), (dict(table=18), BAD),
                     (dict(free=18), BAD), (dict(count=18), BAD), (dict(P=4), UNSUP), (dict(P=48), UNSUP),
                     (dict(P=512), UNSUP), (dict(n=65536), UNSUP), (dict(mp=1 << 25), UNSUP)]:
        assert _tables(lib, **kw) == want, kw
    for name in qsa.Batch._NAMES:
        assert _tables(lib, {name: 18}) == BAD
        assert _tables(lib, {name: None}) == (BAD if name in ("seq_start", "pos_start", "state") else GO)
    assert _tables(lib) == GO and _tables(lib, n=0) == GO and _tables(lib, rows=0) == GO
    assert _tables(lib, cap=0, free=None) == GO and _tables(lib, n=65535) == GO


def test_tables_whose_sums_would_pass_31_bits(lib):
    """Sums of rows and pages stop at 2^31 - 1, which has to lie past every limit, and
    rows are stored in fours from a multiple of 4."""
    for kw in (dict(rows=2 ** 31 - 1), dict(rows=2 ** 30 + 1), dict(cap=2 ** 31 - 1), dict(cap=2 ** 30 + 1)):
        assert _tables(lib, **kw) == UNSUP, kw
    assert _tables(lib, rows=2 ** 30) == GO and _tables(lib, cap=2 ** 30) == GO


def _table(lib, kind=None, n=10, dim=64, theta=1e4, ptr=16, **kw):
    a = dict(factor=2.0, original=4096.0, fast=32.0, slow=1.0, amplitude=1.0)
    a.update(kw)
    c = None if kind is None else ctypes.byref(qsa.RopeScalingC(kind, *a.values()))
    return lib.qsa_rotary_table(vp(ptr), n, dim, theta, c, None)


def test_rotary_table(lib):
    nan, inf = float("nan"), float("inf")
    for kw, want in [(dict(n=-1), BAD), (dict(dim=8), UNSUP), (dict(dim=24), UNSUP), (dict(dim=272), UNSUP),
                     (dict(theta=0.0), BAD), (dict(theta=nan), BAD), (dict(theta=inf), BAD), (dict(ptr=None), BAD),
                     (dict(ptr=24), BAD), (dict(kind=0), BAD), (dict(kind=4), BAD), (dict(kind=1, factor=0.0), BAD),
                     (dict(kind=1, factor=nan), BAD), (dict(kind=2, factor=inf), BAD), (dict(kind=1, amplitude=0.0), BAD),
                     (dict(kind=3, original=0.0), BAD), (dict(kind=3, fast=1.0), BAD), (dict(kind=3, slow=-1.0), BAD),
                     (dict(kind=3, fast=inf), BAD), (dict(kind=2, theta=1e308, factor=1e10), BAD)]:
        assert _table(lib, **kw) == want, kw
    for kind in (None, 1, 2, 3):
        assert _table(lib, kind) == GO
    assert _table(lib, n=0) == qsa.QSA_OK and _table(lib, 1, original=0.0) == GO and _table(lib, dim=256) == GO


def test_rotary_table_of_infinite_angles(lib):
    for kw in (dict(theta=1e-320, dim=256, n=2 ** 20), dict(kind=1, factor=1e-308, n=100), dict(kind=3, factor=1e-308, n=10000),
               dict(kind=2, theta=1e-300, factor=1e-20)):
        assert _table(lib, **kw) == BAD, kw
    assert _table(lib, theta=1e-3) == GO and _table(lib, 1, factor=1e-30) == GO


def _rotary(lib, **kw):
    a = dict(q=16, qs=24 * 256, hq=24, oq=32, oqs=24 * 256, k=16, ks=512, hk=2, ok=32, oks=512, rows=4, D=256, first=0,
             dim=64, layout=0, n=2, ss=16, ps=16, tab=16, n_pos=100)
    a.update(kw)
    return lib.qsa_rotary(vp(a["q"]), a["qs"], a["hq"], vp(a["oq"]), a["oqs"], vp(a["k"]), a["ks"], a["hk"],
                          vp(a["ok"]), a["oks"], a["rows"], a["D"], a["first"], a["dim"], a["layout"], a["n"],
                          vp(a["ss"]), vp(a["ps"]), vp(a["tab"]), a["n_pos"], None)


def test_rotary(lib):
    for kw, want in [(dict(rows=-1), BAD), (dict(n=-1), BAD), (dict(n_pos=0), BAD), (dict(hq=0), BAD), (dict(hk=-1), BAD),
                     (dict(first=-8), BAD), (dict(layout=2), BAD), (dict(D=8), UNSUP), (dict(D=520), UNSUP),
                     (dict(D=528), UNSUP), (dict(D=264), UNSUP), (dict(dim=8), UNSUP), (dict(dim=24), UNSUP),
                     (dict(dim=272, D=512), UNSUP), (dict(first=4), UNSUP), (dict(first=200), UNSUP),
                     (dict(first=2 ** 31 - 8), UNSUP), (dict(n=65536), UNSUP), (dict(hq=4096), UNSUP),
                     (dict(q=None), BAD), (dict(q=24), BAD), (dict(oq=None), BAD), (dict(qs=6136), BAD),
                     (dict(qs=6148), BAD), (dict(oqs=6136), BAD), (dict(k=None), BAD), (dict(ks=504), BAD),
                     (dict(ok=40), BAD), (dict(oks=516), BAD), (dict(ss=None), BAD), (dict(ps=18), BAD),
                     (dict(tab=None), BAD), (dict(tab=24), BAD),
                     (dict(oq=16, oqs=7168), BAD), (dict(ok=16, ks=520), BAD)]:            # in place, strides differ
        assert _rotary(lib, **kw) == want, kw
    assert _rotary(lib, rows=0) == qsa.QSA_OK and _rotary(lib, n=0) == qsa.QSA_OK
    assert _rotary(lib) == GO and _rotary(lib, hk=0, k=None, ok=None) == GO and _rotary(lib, first=192) == GO
    assert _rotary(lib, oq=16, ok=16) == GO and _rotary(lib, layout=1, D=64, qs=1536, ks=128) == GO


def _blocks(lib, cache=None, **kw):
    a = dict(q=16, qs=24 * 256, rows=4, hq=24, n=2, ss=16, ps=16, sel=16, k=8, recent=1, scale=0.0625, out=16, ws=256,
             wsb=1 << 60)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.qsa_block_attention(vp(a["q"]), a["qs"], a["rows"], a["hq"], a["n"], vp(a["ss"]), vp(a["ps"]),
                                   ctypes.byref(c), vp(a["sel"]), a["k"], a["recent"], a["scale"], vp(a["out"]),
                                   vp(a["ws"]), a["wsb"], None)


def test_block_attention(lib):
    for kw, want in [(dict(rows=-1), BAD), (dict(n=-1), BAD), (dict(ss=None), BAD), (dict(ps=18), BAD), (dict(n=3), UNSUP),
                     (dict(cache=_cache(k=None)), BAD), (dict(cache=_cache(dtype=2)), BAD),
                     (dict(cache=_cache(head_dim=64)), UNSUP), (dict(cache=_cache(page_tokens=48)), UNSUP),
                     (dict(q=None), BAD), (dict(q=24), BAD), (dict(out=None), BAD), (dict(out=24), BAD),
                     (dict(qs=6136), BAD), (dict(qs=6148), BAD), (dict(hq=0), BAD), (dict(hq=25), UNSUP),
                     (dict(hq=258, qs=1 << 17), UNSUP), (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD),
                     (dict(scale=2.4e38), BAD), (dict(k=-1), BAD), (dict(recent=-1), BAD),
                     (dict(k=qsa.QSA_MAX_K + 1), UNSUP), (dict(recent=qsa.QSA_MAX_K + 1), UNSUP), (dict(sel=None), BAD),
                     (dict(sel=18), BAD), (dict(cache=_cache(max_pages=(1 << 19) + 1)), UNSUP),
                     (dict(ws=None), qsa.QSA_ERR_WORKSPACE), (dict(wsb=255), qsa.QSA_ERR_WORKSPACE), (dict(ws=128), BAD)]:
        assert _blocks(lib, **kw) == want, kw
    assert _blocks(lib, rows=0) == qsa.QSA_OK and _blocks(lib, n=0) == qsa.QSA_OK
    assert _blocks(lib) == GO and _blocks(lib, k=0, sel=None) == GO and _blocks(lib, hq=256, qs=1 << 16) == GO
    assert _blocks(lib, cache=_cache(max_pages=1 << 19)) == GO
    assert _blocks(lib, cache=_cache(dtype=qsa.QSA_KV_E4M3, k_scale=1, v_scale=3), k=qsa.QSA_MAX_K) == GO


def test_block_attention_workspace():
    n = qsa.block_attention_workspace_bytes(4, 24, 2, 256, 8, 1, 1024)
    assert n >= 256 and n % 256 == 0
    assert qsa.block_attention_workspace_bytes(0, 24, 2, 256, 8, 1, 1024) >= 256


def test_python_checks():
    """The binding names the wrong argument before it calls the library."""
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        qsa.rotary(x, None, i, i[:2], torch.zeros(8, 32))                 # not on a GPU
    with pytest.raises(ValueError):
        qsa.Batch.empty(2, 4, "cpu")
    with pytest.raises(ValueError):
        qsa.RopeScaling("cubic", 2.0)
