"""Host-side refusals of the 8-bit cache's and the page pool's entry points:
they return before anything is launched (no GPU)."""
import ctypes

import pytest

from tree_verification_jsv_b200 import build as jbuild
from tree_verification_jsv_b200 import jsv

INVALID, UNSUPPORTED = jsv.JSV_ERR_INVALID_ARG, jsv.JSV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    jbuild.build()
    return jsv.load()


def batch(**kw):
    base = dict(B=1, Hq=4, Hkv=2, D=128, max_pages_per_req=4, num_pages=4, total_nodes=8, max_nodes=8, max_prefix=32,
                page_table=16, prefix_len=16, node_offsets=16, parent=16)
    base.update(kw)
    return jsv.make_batch(**base)


def cache(**kw):
    base = dict(format="e4m3", num_pages=4, max_pages_per_req=4, k=16, v=16, k_scale=16, v_scale=16, page_table=16)
    base.update(kw)
    return jsv.make_kv8(**base)


def attention(lib, b, c, q=16, k=16, v=16, scale=0.1, out=16, ws=256, nws=1 << 40):
    return lib.jsv_tree_attention_kv8(ctypes.byref(b), ctypes.byref(c), q, k, v, scale, out, ws, nws, None)


def quantize(lib, b, c, k=16, v=16, frm=None, to=16):
    return lib.jsv_kv8_quantize(ctypes.byref(b), ctypes.byref(c), k, v, frm, to, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED), (dict(max_nodes=513), UNSUPPORTED),
    (dict(Hq=6, Hkv=4), INVALID), (dict(B=0), INVALID), (dict(total_nodes=0), INVALID), (dict(parent=None), INVALID),
    (dict(B=40000, total_nodes=40000), UNSUPPORTED)])
def test_batches(lib, kw, code):
    assert attention(lib, batch(**kw), cache()) == code
    assert quantize(lib, batch(**kw), cache()) == code
    assert lib.jsv_tree_attention_kv8_workspace_size(ctypes.byref(batch(**kw)), ctypes.byref(cache())) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(format=2), UNSUPPORTED), (dict(format=-1), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(max_pages_per_req=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(v=24), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(page_table=None), INVALID),
    (dict(num_pages=1 << 27), UNSUPPORTED)])
def test_caches(lib, kw, code):
    assert attention(lib, batch(), cache(**kw)) == code
    assert quantize(lib, batch(), cache(**kw)) == code
    assert lib.jsv_tree_attention_kv8(ctypes.byref(batch()), None, 16, 16, 16, 0.1, 16, 256, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=18), dict(k=8),
                                dict(v=8), dict(out=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf"))])
def test_attention_arguments(lib, kw):
    assert attention(lib, batch(), cache(), **kw) == INVALID


def test_attention_workspace(lib):
    b, c = batch(max_prefix=8192, max_pages_per_req=600), cache()
    need = lib.jsv_tree_attention_kv8_workspace_size(ctypes.byref(b), ctypes.byref(c))
    assert need > 0
    assert attention(lib, b, c, nws=need - 1) == INVALID
    assert attention(lib, b, c, ws=None) == INVALID
    assert attention(lib, b, c, ws=128) == INVALID


def test_quantize_arguments(lib):
    for kw in (dict(k=None), dict(v=None), dict(to=None), dict(k=8), dict(v=8)):
        assert quantize(lib, batch(), cache(), **kw) == INVALID
    assert quantize(lib, batch(B=8193, Hkv=1, Hq=1, total_nodes=8193), cache()) == UNSUPPORTED


def pool(**kw):
    base = dict(num_pages=8, refcount=16)
    base.update(kw)
    return jsv.make_page_pool(**base)


def pool_calls(lib, p, table=16, B=2, width=4, ws=16, nws=1 << 20):
    r = ctypes.byref(p)
    return {
        "alloc": lib.jsv_pages_alloc(r, table, B, width, None, 16, 0, ws, nws, None),
        "fork": lib.jsv_pages_fork(r, table, B, width, 2, 16, 16, 16, 0, 16, 16, ws, nws, None),
        "trim": lib.jsv_pages_trim(r, table, B, width, None, 16, None),
        "compact": lib.jsv_pages_compact(r, table, B, width, 16, 32, 16, 16, 4, 16, ws, nws, None),
    }


@pytest.mark.parametrize("kw,code", [(dict(table=None), INVALID), (dict(B=0), INVALID), (dict(width=0), INVALID),
                                     (dict(B=8193), UNSUPPORTED), (dict(width=1 << 28), UNSUPPORTED)])
def test_pool_tables(lib, kw, code):
    assert set(pool_calls(lib, pool(), **kw).values()) == {code}


@pytest.mark.parametrize("kw", [dict(num_pages=0), dict(refcount=None)])
def test_pools(lib, kw):
    assert set(pool_calls(lib, pool(**kw)).values()) == {INVALID}


@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=24), dict(nws=8)])
def test_pool_workspaces(lib, kw):
    kw = {"ws": 16, "nws": 1 << 20, **kw}
    r, ws = ctypes.byref(pool()), (kw["ws"], kw["nws"], None)
    assert lib.jsv_pages_alloc(r, 16, 2, 4, None, 16, 0, *ws) == INVALID
    assert lib.jsv_pages_fork(r, 16, 2, 4, 2, 16, 16, 16, 0, 16, 16, *ws) == INVALID
    assert lib.jsv_pages_compact(r, 16, 2, 4, 16, 32, 16, 16, 4, 16, *ws) == INVALID


def test_pool_other_arguments(lib):
    r = ctypes.byref(pool())
    assert lib.jsv_pages_workspace_size(8, 2) >= 4 * (8 + 2) and lib.jsv_pages_workspace_size(0, 2) == 0
    assert lib.jsv_pages_alloc(r, 16, 2, 4, None, None, 0, 16, 1 << 20, None) == INVALID
    assert lib.jsv_pages_trim(r, 16, 2, 4, None, None, None) == INVALID
    for at in range(5):
        ptr = [None if i == at else 16 for i in range(5)]
        assert lib.jsv_pages_fork(r, 16, 2, 4, 2, *ptr[:3], 0, *ptr[3:], 16, 1 << 20, None) == INVALID
    assert lib.jsv_pages_fork(r, 16, 2, 4, -1, 16, 16, 16, 0, 16, 16, 16, 1 << 20, None) == INVALID
    assert lib.jsv_pages_fork(r, 16, 2, 4, 8193, 16, 16, 16, 0, 16, 16, 16, 1 << 30, None) == UNSUPPORTED
    assert lib.jsv_pages_fork(r, 16, 2, 4, 0, None, None, None, 0, None, None, None, 0, None) == jsv.JSV_OK
    # compaction: counts in place, too short lists, missing outputs
    assert lib.jsv_pages_compact(r, 16, 2, 4, 16, 16, 16, 16, 4, 16, 16, 1 << 20, None) == INVALID
    assert lib.jsv_pages_compact(r, 16, 2, 4, 16, 32, 16, 16, 3, 16, 16, 1 << 20, None) == INVALID
    assert lib.jsv_pages_compact(r, 16, 2, 4, 16, 32, None, 16, 4, 16, 16, 1 << 20, None) == INVALID
    assert lib.jsv_pages_compact(r, 16, 2, 4, 16, 32, 16, 16, 4, None, 16, 1 << 20, None) == INVALID


def test_copy_arguments(lib):
    p = pool()

    def copy(addr=16, nbytes=64, n_buffers=1, src=16, dst=16, n=3):
        bufs, sizes = (ctypes.c_void_p * 1)(addr), (ctypes.c_int64 * 1)(nbytes)
        return lib.jsv_pages_copy(ctypes.byref(p), bufs, sizes, n_buffers, src, dst, n, None, None)

    for kw in (dict(addr=None), dict(addr=18), dict(nbytes=0), dict(nbytes=6), dict(nbytes=-4), dict(n_buffers=-1),
               dict(src=None), dict(dst=None), dict(n=-1)):
        assert copy(**kw) == INVALID, kw
    assert copy(n=0) == jsv.JSV_OK and copy(n_buffers=0) == jsv.JSV_OK
    assert lib.jsv_pages_copy(ctypes.byref(p), None, None, 1, 16, 16, 3, None, None) == INVALID


def test_status_string_of_an_empty_pool(lib):
    assert "pool" in jsv.status_string(jsv.JSV_ERR_NO_PAGES)
