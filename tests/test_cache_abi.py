"""Host-side checks of the 4-bit cache's and the pages' calls: refusals before anything
touches a device, empty calls, workspace sizes.  No call here reaches the GPU."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from gated_deltanet_linear_06_gb300 import build as gbuild

FAKE, WS = 0x10000, 0x100000          # aligned, never dereferenced on these paths
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _store(L, dims, **kw):
    a = dict(page=64, n_pages=10, tokens=4, k=FAKE, k_st=512, k_sh=256, v=FAKE, v_st=512, v_sh=256, slot=FAKE,
             cache=FAKE, status=None, stream=None)
    a.update(kw)
    return L.gdn_kv4_store(_ref(dims), *a.values())


def _load(L, dims, **kw):
    a = dict(page=64, n_pages=10, tokens=4, slot=FAKE, cache=FAKE, k_out=FAKE, v_out=FAKE, dtype=0, status=None,
             stream=None)
    a.update(kw)
    return L.gdn_kv4_load(_ref(dims), *a.values())


def _attn(L, dims, **kw):
    a = dict(page=64, n_pages=10, batch=2, steps=1, q=FAKE, cache=FAKE, table=FAKE, width=3, len=FAKE, gate=None,
             g_st=0, g_sh=0, out=FAKE, ws=WS, ws_bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return L.gdn_attn_decode_kv4(_ref(dims), *a.values())


@pytest.mark.parametrize("bad,want", [
    (dict(h_q=0), INVALID), (dict(h_kv=3), INVALID), (dict(d=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(d=512), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(h_q=2048, h_kv=2048), UNSUPPORTED)])
def test_dims_are_checked(L, bad, want):
    d = gdn.make_attn_dims(**bad)
    assert _store(L, d) == want and _load(L, d) == want and _attn(L, d) == want
    assert gdn.gdn_attn_decode_kv4_workspace_bytes(d, 2) == 0 and gdn.gdn_kv4_page_bytes(d, 64) == 0
    assert _store(L, None) == INVALID and _load(L, None) == INVALID and _attn(L, None) == INVALID


@pytest.mark.parametrize("bad,want", [
    (dict(page=0), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(n_pages=-1), INVALID), (dict(n_pages=1 << 25), UNSUPPORTED), (dict(cache=None), INVALID),
    (dict(cache=FAKE + 8), INVALID), (dict(status=FAKE + 2), INVALID)])
def test_cache_is_checked(L, bad, want):
    d = gdn.make_attn_dims()
    assert _store(L, d, **bad) == want and _load(L, d, **bad) == want and _attn(L, d, **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID), (dict(slot=FAKE + 4), INVALID),
    (dict(slot=None, tokens=641), INVALID)])
def test_rows_are_checked(L, bad, want):
    d = gdn.make_attn_dims()
    assert _store(L, d, **bad) == want and _load(L, d, **bad) == want
    for more in (dict(k=FAKE + 2), dict(v=FAKE + 8), dict(k_st=513), dict(k_sh=-8), dict(v_st=4), dict(v_sh=12)):
        assert _store(L, d, **more) == INVALID
    for more in (dict(k_out=FAKE + 8), dict(v_out=FAKE + 4), dict(dtype=2)):
        assert _load(L, d, **more) == INVALID


@pytest.mark.parametrize("bad,want", [
    (dict(batch=-1), INVALID), (dict(batch=1025), UNSUPPORTED), (dict(steps=0), INVALID), (dict(steps=9), UNSUPPORTED),
    (dict(width=-1), INVALID), (dict(width=1 << 26), UNSUPPORTED), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(out=None), INVALID), (dict(table=None), INVALID), (dict(table=FAKE + 4), INVALID), (dict(len=None), INVALID),
    (dict(len=FAKE + 4), INVALID), (dict(n_pages=0), INVALID), (dict(gate=FAKE, g_st=4, g_sh=256), INVALID),
    (dict(gate=FAKE + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=WS + 16), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE)])
def test_attention_refusals(L, bad, want):
    assert _attn(L, gdn.make_attn_dims(), **bad) == want


def test_empty_calls_do_nothing(L):
    d = gdn.make_attn_dims()
    assert _store(L, d, tokens=0, k=None, cache=None) == OK and _store(L, d, k=None, v=None, cache=None) == OK
    assert _load(L, d, tokens=0) == OK and _load(L, d, k_out=None, v_out=None) == OK
    assert _attn(L, d, batch=0, q=None, ws=None) == OK
    assert gdn.gdn_kv4_page_bytes(d, 64) == 64 * 2 * 256 * 9 // 8 and gdn.gdn_kv4_page_bytes(d, 48) == 0
    # 128 rows are the most
    wide = gdn.make_attn_dims(h_q=34, h_kv=2)
    assert gdn.gdn_attn_decode_kv4_workspace_bytes(wide, 1, 7) > 0
    assert gdn.gdn_attn_decode_kv4_workspace_bytes(wide, 1, 8) == 0 and _attn(L, wide, steps=8) == UNSUPPORTED


def _pool(**kw):
    a = dict(n_pages=100, page=64, n_seqs=20, width=10, refs=FAKE, table=FAKE, len=FAKE)
    a.update(kw)
    return gdn.PagePool(*a.values())


def _caches(n=1, base=FAKE, size=1024):
    p = gdn.PageCaches(n, (ctypes.c_void_p * 200)(*[base] * 200), (ctypes.c_size_t * 200)(*[size] * 200))
    return p


def _calls(L, pool, caches=None, ws=WS, ws_bytes=1 << 40, status=None, n=4, seq=FAKE):
    tail = (ws, ws_bytes, status, None)
    p, c = _ref(pool), _ref(caches)
    return {"extend": L.gdn_pages_extend(p, seq, n, 3, FAKE, FAKE, *tail),
            "trim": L.gdn_pages_trim(p, c, seq, n, FAKE, *tail),
            "fork": L.gdn_pages_fork(p, c, FAKE, seq, n, *tail),
            "free": L.gdn_pages_free(p, seq, n, *tail),
            "compact": L.gdn_pages_compact(p, c, FAKE, *tail)}


@pytest.mark.parametrize("bad,want", [
    (dict(n_pages=-1), INVALID), (dict(page=0), INVALID), (dict(n_seqs=-1), INVALID), (dict(width=-1), INVALID),
    (dict(n_seqs=65537), UNSUPPORTED), (dict(n_pages=1 << 25), UNSUPPORTED), (dict(width=1 << 25), UNSUPPORTED)])
def test_pool_is_checked(L, bad, want):
    assert set(_calls(L, _pool(**bad)).values()) == {want}
    assert gdn.gdn_pages_workspace_bytes(_pool(**bad)) == 0
    assert set(_calls(L, None).values()) == {INVALID}


@pytest.mark.parametrize("bad", [dict(refs=None), dict(table=None), dict(len=None), dict(refs=FAKE + 4),
                                 dict(table=FAKE + 8), dict(len=FAKE + 4)])
def test_pool_memory_is_checked(L, bad):
    assert set(_calls(L, _pool(**bad)).values()) == {INVALID}


def test_workspaces_lists_and_status(L):
    need = gdn.gdn_pages_workspace_bytes(_pool())
    assert need > 0
    for ws in (dict(ws=None), dict(ws=WS + 64), dict(ws_bytes=need - 1)):
        assert set(_calls(L, _pool(), **ws).values()) == {WORKSPACE}
    assert set(_calls(L, _pool(), status=FAKE + 2).values()) == {INVALID}
    for bad, want in ((dict(n=-1), INVALID), (dict(n=21), INVALID), (dict(seq=FAKE + 4), INVALID)):
        got = _calls(L, _pool(), ws=None, **bad)
        assert got.pop("compact") == WORKSPACE and set(got.values()) == {want}
    got = _calls(L, _pool(n_seqs=9000), n=8193, ws=None)
    assert got.pop("compact") == WORKSPACE and set(got.values()) == {UNSUPPORTED}
    tail = (WS, 1 << 40, None, None)
    p = _ref(_pool())
    assert L.gdn_pages_extend(p, FAKE, 4, -1, None, FAKE, *tail) == INVALID
    assert L.gdn_pages_extend(p, FAKE, 4, 3, None, None, *tail) == INVALID
    assert L.gdn_pages_extend(p, FAKE, 4, 3, FAKE + 4, FAKE, *tail) == INVALID
    assert L.gdn_pages_trim(p, None, FAKE, 4, None, *tail) == INVALID
    assert L.gdn_pages_fork(p, None, None, FAKE, 4, *tail) == INVALID
    assert L.gdn_pages_fork(p, None, FAKE, None, 4, *tail) == INVALID
    assert L.gdn_pages_compact(p, None, FAKE + 2, *tail) == INVALID


def test_empty_page_calls_do_nothing(L):
    got = _calls(L, _pool(), n=0, ws=None, seq=None)
    assert got.pop("compact") == WORKSPACE and set(got.values()) == {OK}
    assert L.gdn_pages_extend(_ref(_pool()), None, 4, 0, None, None, None, 0, None, None) == OK
    assert L.gdn_pages_compact(_ref(_pool(n_pages=0)), None, None, None, 0, None, None) == OK


@pytest.mark.parametrize("bad,want", [(_caches(-1), INVALID), (_caches(129), UNSUPPORTED), (_caches(2, None), INVALID),
                                      (_caches(2, FAKE + 8), INVALID), (_caches(2, FAKE, 0), INVALID),
                                      (_caches(2, FAKE, 24), INVALID), (_caches(1, FAKE, (1 << 32) + 16), UNSUPPORTED)])
def test_caches_are_checked(L, bad, want):
    got = _calls(L, _pool(), caches=bad, ws=None)
    assert (got["trim"], got["fork"], got["compact"]) == (want,) * 3
    assert L.gdn_pages_copy(_ref(bad), 5, FAKE, _ref(bad), 5, FAKE, 2, None, None) == want


def test_copy_refusals(L):
    def copy(a, b, sp=5, dp=5, s=FAKE, d=FAKE, n=2, status=None):
        return L.gdn_pages_copy(_ref(a), sp, s, _ref(b), dp, d, n, status, None)
    c = _caches(2)
    assert copy(None, c) == INVALID and copy(c, None) == INVALID
    assert copy(c, _caches(1)) == INVALID and copy(c, _caches(2, FAKE, 2048)) == INVALID
    assert copy(c, c, sp=-1) == INVALID and copy(c, c, dp=-1) == INVALID and copy(c, c, n=-1) == INVALID
    assert copy(c, c, s=FAKE + 4) == INVALID and copy(c, c, d=FAKE + 4) == INVALID
    assert copy(c, c, s=None, n=6) == INVALID and copy(c, c, d=None, n=6) == INVALID
    assert copy(c, c, status=FAKE + 1) == INVALID
    assert copy(c, c, n=0) == OK and copy(_caches(0), _caches(0)) == OK


def test_python_refusals():
    d = gdn.make_attn_dims()
    t = torch.zeros(3, 2, 4, 18 * 256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        gdn.gdn_kv4_store(d, None, None, t)                      # not on a GPU
    with pytest.raises(ValueError):
        gdn.gdn_kv4_store(d, None, None, t[:, :1])
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.make_page_pool(i, i, i, 16)
    with pytest.raises(ValueError):
        gdn.make_page_pool(i, i.view(4, 1), i, 16)               # not on a GPU
    with pytest.raises(ValueError):
        gdn.make_page_caches([t, t[:2]])


def test_library_exports_the_calls(L):
    for name in ("gdn_kv4_page_bytes", "gdn_kv4_store", "gdn_kv4_load", "gdn_attn_decode_kv4",
                 "gdn_attn_decode_kv4_workspace_bytes", "gdn_pages_workspace_bytes", "gdn_pages_extend",
                 "gdn_pages_trim", "gdn_pages_fork", "gdn_pages_free", "gdn_pages_compact", "gdn_pages_copy"):
        assert hasattr(L, name)
