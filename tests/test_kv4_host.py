"""Refusals of the 4-bit cache's calls and of rotation by several axes (no GPU)."""
import numpy as np
import pytest

from heterogeneous_compressed_kv_gb300 import kvpool as K

P16 = 1 << 20  # plausible, aligned addresses that nothing reads
FAR = 1 << 30


def heads(n=2, d=64, data=P16, ts=None, hs=None):
    return (data or 0, n * d if ts is None else ts, d if hs is None else hs, n, 0)


def i64(*x):
    return np.array(x, np.int64)


def cache(pages=FAR, n_pages=10, table=FAR + (1 << 24), stride=4, rows=3, width=4, hk=2, d=64, page=64, ks=1.0, vs=1.0):
    return K._KV4.pack(pages or 0, n_pages, table or 0, stride, rows, width, hk, d, page, ks, vs, 0)


def test_page_bytes():
    f = K.lib().kvpool_kv4_page_bytes
    assert f(2, 64, 16) == 2 * 16 * (64 + 8) and f(16, 128, 256) == 16 * 256 * (128 + 16)
    for bad in [(0, 64, 16), (1025, 64, 16), (2, 96, 16), (2, 64, 8), (2, 64, 48), (2, 64, 2048), (2, 64, 0), (-1, 64, 16)]:
        assert f(*bad) == K.ERR_INVALID_ARG
        with pytest.raises(K.KvpoolError):
            K.kv4_page_bytes(*bad)


def move(which, start=(0, 5), n=(3, 70), dtype=K.BF16, k=None, v=None, rows=100, segs=None, **kw):
    a, b = i64(*start), i64(*n)
    k, v = k or heads(data=P16), v or heads(data=P16 + (1 << 22))
    f = getattr(K.lib(), "kvpool_kv4_" + which)
    return f(cache(**kw), dtype, K._HEADS.pack(*k), K._HEADS.pack(*v), rows, a.size if segs is None else segs, a.ctypes.data,
             b.ctypes.data, None)


BAD_CACHE = [dict(pages=FAR + 8), dict(n_pages=-1), dict(n_pages=1 << 31), dict(stride=-1), dict(rows=1), dict(rows=-1), dict(width=-1),
             dict(table=FAR + 2), dict(hk=0), dict(d=96), dict(page=24), dict(ks=0.0), dict(ks=-1.0), dict(ks=3.0), dict(vs=float("nan")),
             dict(vs=float("inf")), dict(vs=2.0 ** 17), dict(ks=2.0 ** -17), dict(width=1 << 25)]


@pytest.mark.parametrize("which", ["store", "load"])
@pytest.mark.parametrize("bad", BAD_CACHE + [
    dict(start=(0, -1)), dict(n=(3, -1)), dict(n=(3, 252)), dict(start=(254, 0)), dict(start=(1 << 62, 0)), dict(n=(3, 1 << 62)),
    dict(rows=72), dict(rows=-1), dict(dtype=K.FP8_E4M3), dict(segs=-1), dict(k=heads(3)), dict(v=heads(1)), dict(k=heads(ts=65)),
    dict(k=heads(data=P16 + 4)), dict(k=heads(data=None)), dict(pages=None), dict(table=None)])
def test_moves_refuse(which, bad):
    assert move(which, **bad) == K.ERR_INVALID_ARG


def test_loads_refuse_outputs_that_meet():
    assert move("load", v=heads(data=P16)) == K.ERR_INVALID_ARG
    assert move("load", k=heads(hs=0)) == K.ERR_INVALID_ARG
    assert move("load", k=heads(ts=64, hs=64)) == K.ERR_INVALID_ARG


def test_moves_without_work():
    for which in ("store", "load"):
        assert move(which, start=(), n=()) == K.OK
        assert move(which, n=(0, 0), start=(9, 256)) == K.OK
        assert move(which, n=(0, 0), pages=None, table=None, k=heads(data=None), v=heads(data=None)) == K.OK


def attend(q_len=(1, 2), k_len=(100, 200), dtype=K.BF16, scale=0.125, q=None, out=None, rows=10, lse=0, w=0, ws=1 << 20, wh=1 << 10,
           decay=1.0, segs=None, space=None, space_bytes=0, work_too=True, **kw):
    a, b = i64(*q_len), i64(*k_len)
    q = q or heads(4)
    out = out or heads(4, data=P16 + (1 << 22))
    args = cache(**kw) + K._KV4_ARGS.pack(dtype, scale, *q, *out, rows, lse, w, ws, wh, decay, 0)
    call = (args, a.size if segs is None else segs, a.ctypes.data, b.ctypes.data)
    got = K.lib().kvpool_kv4_attend(*call, space, space_bytes, None)
    if work_too:
        assert K.lib().kvpool_kv4_workspace(*call) == got
    return got


@pytest.mark.parametrize("bad", BAD_CACHE + [
    dict(q_len=(1, -1)), dict(k_len=(1, -1)), dict(k_len=(1, 257)), dict(k_len=(1, 1 << 62)), dict(q_len=(1, 1 << 62)), dict(rows=2),
    dict(rows=-1), dict(dtype=K.FP8_E4M3), dict(scale=float("inf")), dict(scale=float("nan")), dict(decay=float("nan")), dict(segs=-1),
    dict(q=heads(3)), dict(q=heads(1)), dict(q=heads(34), out=heads(34, data=FAR * 2)), dict(out=heads(2, data=FAR * 2)),
    dict(q=heads(4, data=P16 + 2)), dict(q=heads(4, ts=4)), dict(out=heads(4, data=FAR * 2, hs=0)), dict(q=heads(4, data=None)),
    dict(out=heads(4, data=None)), dict(pages=None), dict(table=None), dict(n_pages=0),
    dict(w=P16 + 2), dict(w=P16, wh=199), dict(w=P16, ws=199), dict(w=P16, ws=1 << 9, wh=500), dict(w=P16, ws=-1),
    dict(w=P16, q_len=(1, 33))])
def test_attend_refuses(bad):
    assert attend(**bad) == K.ERR_INVALID_ARG


def test_outputs_on_the_cache_are_refused():
    on = heads(4, data=FAR + 4096)
    assert attend(out=on, work_too=False) == K.ERR_INVALID_ARG and attend(lse=FAR - 16, work_too=False) == K.ERR_INVALID_ARG
    assert attend(out=heads(4, data=FAR + (1 << 24) + 32), work_too=False) == K.ERR_INVALID_ARG  # the table
    assert attend(w=P16, space=FAR + 256, space_bytes=1 << 20, work_too=False) == K.ERR_INVALID_ARG
    assert move("store", k=heads(data=FAR + 64)) == K.ERR_INVALID_ARG and move("load", v=heads(data=FAR - 128)) == K.ERR_INVALID_ARG
    assert evict(index=FAR + 64) == K.ERR_INVALID_ARG


def test_attend_refuses_an_output_on_its_queries():
    assert attend(out=heads(4, data=P16 + 128), work_too=False) == K.ERR_INVALID_ARG
    assert attend(out=heads(4, data=P16, ts=512), q=heads(4, ts=256), work_too=False) == K.ERR_INVALID_ARG


def test_attend_without_work():
    assert attend(q_len=(), k_len=()) == K.OK
    assert attend(q_len=(0, 0), pages=None, table=None, q=heads(4, data=None), out=heads(4, data=None)) == K.OK


def evict(k_len=(100, 200), keep=50, sink=4, recent=8, out=FAR * 4, ostride=4, orows=3, owidth=4, w=P16, ws=1 << 12, wh=1 << 10,
          ow=FAR * 3, ows=1 << 12, owh=1 << 10, index=FAR * 5, wide=60, segs=None, **kw):
    a = i64(*k_len)
    args = cache(**kw) + K._KV4_EVICT.pack(out or 0, ostride, orows, owidth, w or 0, ws, wh, ow or 0, ows, owh, index or 0, wide, keep, sink,
                                           recent)
    return K.lib().kvpool_kv4_evict(args, a.size if segs is None else segs, a.ctypes.data, None)


@pytest.mark.parametrize("bad", BAD_CACHE + [
    dict(k_len=(1, -1)), dict(k_len=(1, 257)), dict(k_len=(1, 1 << 62)), dict(keep=0), dict(keep=-1), dict(sink=-1), dict(recent=-1),
    dict(sink=51), dict(sink=40, recent=11), dict(sink=2147483647, recent=2147483647), dict(out=None), dict(out=FAR + 2), dict(ostride=-1),
    dict(orows=1), dict(owidth=0), dict(owidth=-1), dict(w=None), dict(w=P16 + 2), dict(ws=-1), dict(wh=-1), dict(ow=P16),
    dict(ow=P16 + 4 * 5000), dict(ow=FAR * 3 + 1), dict(ows=59), dict(ows=1 << 9, owh=500), dict(owh=59), dict(ows=-1), dict(owh=-1), dict(wide=49), dict(index=None), dict(index=FAR + 1),
    dict(segs=-1), dict(n_pages=0), dict(pages=None), dict(table=None)])
def test_evict_refuses(bad):
    assert evict(**bad) == K.ERR_INVALID_ARG


def test_evict_without_segments():
    assert evict(k_len=()) == K.OK


def test_structures_have_the_header_s_sizes():
    assert K._KV4.size == 64
    assert len(cache()) + K._KV4_ARGS.size == 64 + 8 + 64 + 8 + 16 + 16 + 8
    assert len(cache()) + K._KV4_EVICT.size == 64 + 24 + 24 + 24 + 8 + 16


def axes(n_axes=3, ax=bytes([0] * 8 + [1] * 12 + [2] * 12), rot=64, T=0, pos=P16):
    q = K._HEADS.pack(*heads(4))
    return K.lib().kvpool_qk_norm_rope_axes(K.BF16, 64, T, q, q, q, q, None, None, 1e-6, rot, 0, P16, pos, n_axes, ax, None)


@pytest.mark.parametrize("bad", [dict(n_axes=0), dict(n_axes=9), dict(n_axes=-1), dict(n_axes=2), dict(ax=None),
                                 dict(ax=bytes([3] + [0] * 31)), dict(ax=bytes([0] * 31 + [255])), dict(pos=None, T=2)])
def test_axes_refuse(bad):
    assert axes(**bad) == K.ERR_INVALID_ARG


def test_axes_without_work():
    assert axes() == K.OK
    assert axes(n_axes=1, ax=None) == K.OK
    assert axes(rot=0, ax=None) == K.OK
