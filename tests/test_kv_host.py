"""K/V cache entry points on a machine without a GPU: what they refuse before
any launch."""
import ctypes

import pytest
import torch

from block_sparse_attention_select_gb300 import build as qbuild
from block_sparse_attention_select_gb300 import qsa

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def _cache(**kw):
    a = dict(k=16, v=16, k_scale=None, v_scale=None, dtype=qsa.QSA_KV_FP16, num_pages=4, page_tokens=64, hkv=2,
             head_dim=256, block_table=16, num_reqs=2, max_pages=4)
    a.update(kw)
    return qsa.KVCacheC(*a.values())


def _store(lib, cache=None, fn="qsa_kv_store", **kw):
    a = dict(k=16, ks=512, v=16, vs=512, rows=4, n=2, ss=16, ps=16)
    a.update(kw)
    c = _cache() if cache is None else cache
    return getattr(lib, fn)(vp(a["k"]), a["ks"], vp(a["v"]), a["vs"], a["rows"], a["n"], vp(a["ss"]), vp(a["ps"]),
                            ctypes.byref(c), None)


def _attend(lib, cache=None, **kw):
    a = dict(q=16, qs=24 * 256, rows=4, hq=24, n=2, ss=16, ps=16, window=0, scale=0.0625, out=16, ws=256,
             wsb=1 << 40)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.qsa_chunk_attention(vp(a["q"]), a["qs"], a["rows"], a["hq"], a["n"], vp(a["ss"]), vp(a["ps"]),
                                   ctypes.byref(c), a["window"], a["scale"], vp(a["out"]), vp(a["ws"]), a["wsb"], None)


CALLS = [lambda lib, **kw: _store(lib, **kw), lambda lib, **kw: _store(lib, fn="qsa_kv_load", **kw), _attend]


@pytest.mark.parametrize("call", CALLS, ids=["store", "load", "attend"])
def test_refusals_shared_by_the_calls(lib, call):
    bad, unsup = qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_UNSUPPORTED
    for kw, want in [
            (dict(rows=-1), bad), (dict(n=-1), bad), (dict(ss=None), bad), (dict(ps=None), bad),
            (dict(ss=18), bad), (dict(ps=18), bad), (dict(n=3), unsup),     # more requests than the block table has
            (dict(cache=_cache(k=None)), bad), (dict(cache=_cache(v=None)), bad), (dict(cache=_cache(k=24)), bad),
            (dict(cache=_cache(v=24)), bad), (dict(cache=_cache(block_table=None)), bad),
            (dict(cache=_cache(block_table=18)), bad), (dict(cache=_cache(num_pages=0)), bad),
            (dict(cache=_cache(hkv=0)), bad), (dict(cache=_cache(num_reqs=0)), bad),
            (dict(cache=_cache(max_pages=0)), bad), (dict(cache=_cache(dtype=2)), bad),
            (dict(cache=_cache(dtype=qsa.QSA_KV_E4M3)), bad),               # no scales
            (dict(cache=_cache(k_scale=16, v_scale=16)), bad),              # scales of an FP16 cache
            (dict(cache=_cache(head_dim=64)), unsup), (dict(cache=_cache(head_dim=192)), unsup),
            (dict(cache=_cache(page_tokens=4)), unsup), (dict(cache=_cache(page_tokens=48)), unsup),
            (dict(cache=_cache(page_tokens=512)), unsup), (dict(cache=_cache(hkv=1025)), unsup),
            (dict(cache=_cache(num_pages=1 << 25)), unsup), (dict(cache=_cache(max_pages=1 << 25)), unsup)]:
        assert call(lib, **kw) == want, kw
    assert call(lib, rows=0) == qsa.QSA_OK and call(lib, n=0) == qsa.QSA_OK
    assert call(lib) == qsa.QSA_ERR_NO_DEVICE
    assert call(lib, cache=_cache(dtype=qsa.QSA_KV_E4M3, k_scale=1, v_scale=3)) == qsa.QSA_ERR_NO_DEVICE


@pytest.mark.parametrize("fn", ["qsa_kv_store", "qsa_kv_load"])
def test_row_arrays(lib, fn):
    for kw in (dict(k=None), dict(v=None), dict(k=24), dict(v=24), dict(ks=511), dict(ks=504), dict(ks=516),
               dict(vs=504), dict(vs=513)):
        assert _store(lib, fn=fn, **kw) == qsa.QSA_ERR_INVALID_ARG, kw
    assert _store(lib, fn=fn, ks=520, vs=7168) == qsa.QSA_ERR_NO_DEVICE


def test_attention_refusals(lib):
    bad, unsup = qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_UNSUPPORTED
    for kw, want in [
            (dict(q=None), bad), (dict(q=24), bad), (dict(out=None), bad), (dict(out=24), bad), (dict(qs=6136), bad),
            (dict(qs=6148), bad), (dict(hq=0), bad), (dict(hq=25), unsup), (dict(window=-1), bad),
            (dict(scale=0.0), bad), (dict(scale=float("nan")), bad), (dict(scale=float("inf")), bad),
            (dict(hq=258, qs=1 << 17), unsup),                            # 129 query heads per KV head
            (dict(ws=None), qsa.QSA_ERR_WORKSPACE), (dict(wsb=255), qsa.QSA_ERR_WORKSPACE), (dict(ws=128), bad)]:
        assert _attend(lib, **kw) == want, kw
    assert _attend(lib, hq=256, qs=1 << 16) == qsa.QSA_ERR_NO_DEVICE
    n = qsa.chunk_attention_workspace_bytes(4, 24, 2, 256)
    assert n >= 256 and n % 256 == 0


def test_python_checks():
    """The binding names the wrong argument before it calls the library."""
    table = torch.zeros(2, 4, dtype=torch.int32)
    k = torch.zeros(8, 16, 2, 128, dtype=torch.float16)
    with pytest.raises(TypeError):
        qsa.KVCache(k.float(), k.float(), table)
    with pytest.raises(ValueError):                                       # not on a GPU
        qsa.KVCache(k, k, table)
    code = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        qsa.KVCache(code, code, table)
