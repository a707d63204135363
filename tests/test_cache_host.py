"""Refusals of the cache entry points, on the host before anything is enqueued."""
import ctypes

import pytest
import torch
from hypothesis import HealthCheck, given, settings
from hypothesis import strategies as st

import mrope_qk_norm_b200 as qkr

BASE = 1 << 36
E, U = 1, 2
ptrs = st.one_of(st.just(0), st.integers(0, 1 << 24).map(lambda o: BASE + o))
small = st.integers(-3, 300)
wide = st.one_of(small, st.integers(-(1 << 33), 1 << 33))
big = st.one_of(st.integers(0, 64).map(lambda x: 64 * x), st.integers(-(1 << 40), 1 << 40))

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="an accepted call would launch on the fake addresses")


def _plane(i, row, page=16, heads=2):
    return qkr.CachePlane(BASE + (i << 30), page * heads * row, heads * row, row)


def _cache(fmt=qkr.CACHE_BF16, D=64, page=16, pages=8, heads=2, **kw):
    c = qkr.CacheDesc(format=fmt, page_size=page, n_pages=pages, Hkv=heads, D=D)
    row, sc = (2 * D, 0) if fmt == qkr.CACHE_BF16 else (D // 2, D // 16)
    c.k, c.v = _plane(0, row, page, heads), _plane(1, row, page, heads)
    if sc:
        c.k_scale, c.v_scale = _plane(2, sc, page, heads), _plane(3, sc, page, heads)
    for k, v in kw.items():
        obj, _, name = k.partition("__")
        setattr(getattr(c, obj), name, v)
    return c


def _attend(cache=None, **kw):
    a = dict(q=BASE + (4 << 30), out=BASE + (5 << 30), lse=0, T=3, Hq=4, qts=256, qhs=64, ots=256,
             table=BASE + (6 << 30), tstride=8, lens=BASE + (7 << 30), cu=BASE + (8 << 30), B=2,
             max_q=2, max_len=128, scale=0.125, window=0, sink=0, ws=BASE + (9 << 30),
             wsb=1 << 28)
    a.update(kw)
    c = _cache() if cache is None else cache
    return qkr.lib().cache_attention(None, ctypes.byref(c), *a.values())


def _rows(get=False, cache=None, k=BASE + (4 << 30), v=BASE + (5 << 30), idx=BASE + (6 << 30), T=4,
          kts=128, vts=128):
    c = _cache(qkr.CACHE_Q4) if cache is None else cache
    fn = qkr.lib().cache_get_rows_q4 if get else qkr.lib().cache_set_rows_q4
    return fn(None, ctypes.byref(c), k, v, idx, T, kts, vts)


def _message():
    return qkr.lib().qkr_last_error().decode()


def test_a_valid_call_passes_validation():
    # it fails only for want of a device
    assert _attend() == qkr.QKR_ERR_CUDA
    assert _attend(_cache(qkr.CACHE_Q4)) == qkr.QKR_ERR_CUDA
    assert _rows() == qkr.QKR_ERR_CUDA and _rows(get=True) == qkr.QKR_ERR_CUDA


@pytest.mark.parametrize("status,kw", [
    (E, dict(q=0)), (E, dict(out=0)), (E, dict(table=0)), (E, dict(lens=0)), (E, dict(cu=0)),
    (E, dict(T=-1)), (E, dict(B=-1)), (E, dict(max_q=-1)), (E, dict(max_len=-1)),
    (E, dict(Hq=3)), (E, dict(Hq=0)), (E, dict(window=-1)), (E, dict(sink=-1)),
    (E, dict(scale=float("nan"))), (E, dict(scale=float("inf"))),
    (E, dict(max_len=129)), (E, dict(tstride=-1)),
    (U, dict(q=BASE + 8)), (U, dict(out=BASE + (5 << 30) + 8)), (U, dict(lens=BASE + (7 << 30) + 2)),
    (U, dict(qts=252)), (U, dict(qhs=32)), (U, dict(qts=-256)), (U, dict(ots=128)), (U, dict(ots=260)),
    (U, dict(T=1 << 30)), (U, dict(max_len=(1 << 29) + 1, tstride=1 << 30)), (U, dict(B=(1 << 16) + 1)),
])
def test_attention_refusals(status, kw):
    assert _attend(**kw) == status, _message()
    assert _message()


@pytest.mark.parametrize("status,kw", [
    (E, dict(fmt=2)), (U, dict(D=60)), (U, dict(D=136)), (U, dict(D=0)), (U, dict(page=8)),
    (U, dict(page=24)), (E, dict(pages=0)), (E, dict(heads=0)),
    (U, dict(fmt=qkr.CACHE_Q4, D=96)), (U, dict(fmt=qkr.CACHE_Q4, D=32)),
    (E, dict(k__base=0)), (U, dict(v__base=BASE + 8)), (U, dict(k__row_stride=250)),
    (U, dict(k__row_stride=264)), (U, dict(v__head_stride=0)), (U, dict(k__page_stride=-4096)),
    (U, dict(k__page_stride=1 << 32)), (U, dict(v__row_stride=1 << 32)), (U, dict(k__head_stride=1 << 39)),
    (E, dict(fmt=qkr.CACHE_Q4, k_scale__base=0)), (U, dict(fmt=qkr.CACHE_Q4, v_scale__base=BASE + 2)),
])
def test_cache_refusals(status, kw):
    c = _cache(**kw)
    assert _attend(c) == status, _message()
    if kw.get("fmt") == qkr.CACHE_Q4:
        assert _rows(cache=c) == status and _rows(get=True, cache=c) == status


def test_overlaps_are_refused():
    assert _attend(out=BASE + (4 << 30)) == U               # q
    assert _attend(out=BASE + (1 << 30) + 4096) == U        # the cache
    assert _attend(lse=BASE + (5 << 30) + 64) == U          # out
    assert _attend(out=BASE + (6 << 30) - 16) == U          # the page table
    assert _rows(k=BASE + 1024) == U and _rows(idx=BASE + (1 << 30)) == U
    assert _rows(get=True, v=BASE + (4 << 30) + 16) == U    # the other output
    assert _rows(get=True, idx=BASE + (4 << 30)) == U


def test_row_refusals():
    for get in (False, True):
        assert _rows(get, k=0) == E and _rows(get, v=0) == E and _rows(get, idx=0) == E
        assert _rows(get, T=-1) == E and _rows(get, T=1 << 31) == U
        assert _rows(get, k=BASE + 8) == U and _rows(get, idx=BASE + (6 << 30) + 4) == U
        assert _rows(get, kts=64) == U and _rows(get, vts=132) == U
        assert _rows(get, cache=_cache()) == E               # not a 4-bit cache
        assert _rows(get, T=0, k=0, v=0, idx=0) == qkr.QKR_OK
        assert qkr.last_launch()["launches"] == 0


def test_empty_calls_enqueue_nothing():
    for kw in (dict(T=0), dict(B=0), dict(max_q=0)):
        assert _attend(**kw, q=0, out=0, lens=0, cu=0, table=0, ws=0) == qkr.QKR_OK
        assert qkr.last_launch()["launches"] == 0


@settings(max_examples=500, deadline=None, suppress_health_check=list(HealthCheck))
@given(fmt=st.integers(-1, 2), page=st.integers(-16, 1 << 17), pages=st.integers(-2, 1 << 33),
       heads=st.integers(-1, 70), D=st.integers(-8, 300), bases=st.lists(ptrs, min_size=4, max_size=4),
       strides=st.lists(big, min_size=12, max_size=12), args=st.lists(ptrs, min_size=7, max_size=7),
       T=wide, Hq=small, ss=st.lists(big, min_size=4, max_size=4), B=wide, mq=wide, ml=wide,
       scale=st.floats(allow_nan=True, allow_infinity=True), w=big, sink=big, wsb=big)
def test_fuzz(fmt, page, pages, heads, D, bases, strides, args, T, Hq, ss, B, mq, ml, scale, w, sink,
              wsb):
    """Any sizes, strides and pointers come back as a status code with a message."""
    c = qkr.CacheDesc(format=fmt, page_size=page, n_pages=pages, Hkv=heads, D=D)
    c.k, c.v, c.k_scale, c.v_scale = (qkr.CachePlane(bases[i], *strides[3 * i:3 * i + 3])
                                      for i in range(4))
    L, n = qkr.lib(), ctypes.c_int64(0)
    calls = [L.cache_attention(None, ctypes.byref(c), args[0], args[1], args[2], T, Hq, ss[0], ss[1],
                               ss[2], args[3], ss[3], args[4], args[5], B, mq, ml, scale, w, sink,
                               args[6], wsb),
             L.cache_set_rows_q4(None, ctypes.byref(c), args[0], args[1], args[2], T, ss[0], ss[1]),
             L.cache_get_rows_q4(None, ctypes.byref(c), args[0], args[1], args[2], T, ss[0], ss[1]),
             L.cache_attention_workspace(ctypes.byref(c), T, Hq, B, mq, ml, w, sink,
                                         ctypes.byref(n))]
    for status in calls:
        assert status in (qkr.QKR_OK, E, U, qkr.QKR_ERR_CUDA)


def test_workspace_refusals():
    n = ctypes.c_int64(-1)
    c = _cache()

    def need(T=3, Hq=4, B=2, mq=2, ml=128, w=0, s=0, cache=c, out=ctypes.byref(n)):
        return qkr.lib().cache_attention_workspace(ctypes.byref(cache), T, Hq, B, mq, ml, w, s, out)
    assert need(out=None) == E and need(Hq=5) == E and need(T=-1) == E and need(w=-1) == E
    assert need(cache=_cache(fmt=7)) == E
    assert need(T=0) == qkr.QKR_OK and n.value == 0


def test_the_descriptor_is_no_cycle():
    """Dropping a descriptor frees the cache tensors at once, without the collector."""
    import gc
    import weakref
    d = _cache()
    d._keep = keep = type("T", (), {})()
    r = weakref.ref(keep)
    gc.disable()
    try:
        _attend(d)
        del d, keep
        assert r() is None
    finally:
        gc.enable()
