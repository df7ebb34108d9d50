"""Refusals and host parts of the entry points without a pool (no GPU)."""
import numpy as np
import pytest

from heterogeneous_compressed_kv_gb300 import kvpool as K

P16 = 1 << 20  # a plausible, aligned address that nothing reads


def heads(n=4, d=64, data=P16, ts=None, hs=None):
    return (data or 0, n * d if ts is None else ts, d if hs is None else hs, n, 0)


def table(rot, f):
    f = np.ascontiguousarray(f, np.float64)
    out = np.zeros(max(rot // 2, 1), np.uint64)
    return K.lib().kvpool_rope_table(rot, f.ctypes.data, out.ctypes.data), out


def test_rope_table_is_the_fraction_of_a_turn():
    rot = 128
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    rc, t = table(rot, f)
    assert rc == K.OK
    # a double's half step (2^-53 relative) of f / (2 pi) < 1, twice (quotient, 2 pi itself)
    got = t.astype(np.longdouble) / np.longdouble(2) ** 64
    want = f.astype(np.longdouble) / (2 * np.longdouble(np.pi))
    assert np.max(np.abs(got - want)) <= 2.0 ** -52


def test_rope_table_whole_turns_and_negative_frequencies():
    rc, t = table(16, [2 * np.pi, -0.25 * 2 * np.pi, 0.0, 1e-30, -1e-30, 3.5 * 2 * np.pi, 1.0, -1.0])
    assert rc == K.OK
    turns = t.astype(np.float64) / 2.0 ** 64
    assert turns[0] in (0.0,) and turns[1] == 0.75 and turns[2] == 0.0 and turns[5] == 0.5
    assert int(t[6]) + int(t[7]) in range(2 ** 64 - 4096, 2 ** 64 + 4097)  # f and -f are a whole turn together
    assert t[4] == 0


@pytest.mark.parametrize("rot", [-16, 8, 24, 272])
def test_rope_table_refuses_sizes(rot):
    assert table(rot, np.ones(max(rot // 2, 1)))[0] == K.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_rope_table_refuses_frequencies(bad):
    assert table(16, [1, 1, 1, 1, 1, 1, 1, bad])[0] == K.ERR_INVALID_ARG


def rope(dtype=K.BF16, d=64, T=2, q=None, k=None, qo=None, ko=None, eps=1e-6, rot=64, inter=0, tab=P16, pos=P16):
    q, k = q or heads(), k or heads()
    qo, ko = qo or q, ko or k
    q, k, qo, ko = (K._HEADS.pack(*x) for x in (q, k, qo, ko))
    return K.lib().kvpool_qk_norm_rope(dtype, d, T, q, k, qo, ko, None, None, eps, rot, inter, tab, pos, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=K.FP8_E4M3), dict(d=0), dict(d=60), dict(d=264), dict(rot=-16), dict(rot=24), dict(rot=128), dict(T=-1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(inter=2), dict(tab=None), dict(pos=None),
    dict(q=heads(data=P16 + 2)), dict(q=heads(ts=257)), dict(k=heads(hs=68)), dict(k=heads(data=None)),
    dict(q=heads(n=-1)), dict(qo=heads(n=3)), dict(q=heads(n=70000)), dict(qo=heads(data=None))])
def test_rope_refuses(bad):
    assert rope(**bad) == K.ERR_INVALID_ARG


def test_rope_without_work():
    assert rope(T=0) == K.OK
    none = heads(n=0)
    assert rope(q=none, k=none) == K.OK


def window(q_len, k_start, k_len, n=None, ws=None, ws_bytes=0, **kw):
    a = K._WINDOW_ARGS.pack(kw.get("dtype", K.BF16), kw.get("d", 64), *kw.get("q", heads(8)), *kw.get("k", heads(4)),
                            *kw.get("v", heads(4)), *kw.get("out", heads(8)), kw.get("q_rows", 100), kw.get("kv_rows", 1000), 0,
                            kw.get("window", 16), kw.get("sink", 0), kw.get("scale", 0.125), 0)
    ql, ks, kl = (np.array(x, np.int64) for x in (q_len, k_start, k_len))
    call = (a, ql.size if n is None else n, ql.ctypes.data, ks.ctypes.data, kl.ctypes.data)
    got = K.lib().kvpool_window_attend(*call, ws, ws_bytes, None)
    assert K.lib().kvpool_window_workspace(*call) == (got if got else 0)
    return got


@pytest.mark.parametrize("bad", [
    dict(dtype=K.FP8_E4M3), dict(d=96), dict(q=heads(3)), dict(q=heads(6)), dict(q=heads(68)), dict(out=heads(4)),
    dict(v=heads(8)), dict(k=heads(0), v=heads(0)), dict(window=-1), dict(sink=-1), dict(scale=float("nan")),
    dict(q_rows=1), dict(q_rows=-1), dict(q_rows=1 << 31), dict(kv_rows=1 << 31), dict(q=heads(8, data=None)),
    dict(k=heads(4, data=None)), dict(v=heads(4, data=P16 + 8)), dict(k=heads(4, ts=257)), dict(out=heads(8, hs=-64))])
def test_window_refuses_arguments(bad):
    assert window([2], [0], [5], **bad) == K.ERR_INVALID_ARG


@pytest.mark.parametrize("seg", [([-1], [0], [5]), ([1], [0], [-1]), ([1], [-1], [5]), ([1], [996], [5]),
                                 ([1], [1 << 40], [5]), ([60, 60], [0, 0], [60, 60]), ([1], [0], [(1 << 30) + 1])])
def test_window_refuses_segments(seg):
    assert window(*seg) == K.ERR_INVALID_ARG


def test_window_without_work():
    assert window([], [], []) == K.OK
    assert window([0, 0], [0, 5], [10, 0]) == K.OK
    assert window([1], [0], [5], n=-1) == K.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(ts=0), dict(hs=0), dict(ts=32), dict(hs=56)])
def test_outputs_that_share_values_are_refused(bad):
    assert rope(qo=heads(**bad)) == K.ERR_INVALID_ARG
    assert rope(ko=heads(**bad)) == K.ERR_INVALID_ARG
    assert window([2], [0], [5], out=heads(8, **bad)) == K.ERR_INVALID_ARG


def test_shared_decode_refuses_what_is_not_shared():
    from tests.test_abi_host import base_workload, cfg_of
    p = K.Pool(cfg_of(base_workload(layer_kinds=[K.HCA])))
    a, b, c = (p.alloc_request() for _ in range(3))
    buf = np.zeros(16, np.float32).ctypes.data

    def call(ids, n_shared, layer=0):
        return p.decode_attend_shared(layer, ids, n_shared, buf, buf, 0, buf, stream=0, check=False)

    p.append([a], [600], 1, 1, 1, stream=0)
    p.append([c], [600], 1, 1, 1, stream=0)
    p.share_prefix(b, a, 256, 1, 1, stream=0)
    p.append([b], [300], 1, 1, 1, stream=0)
    assert call([a, b], 256) == K.ERR_INVALID_ARG and "no device" in p.last_error()  # shared: only the device is missing
    assert call([b, a, b], 128) == K.ERR_INVALID_ARG and "no device" in p.last_error()
    assert call([a], 512) == K.ERR_INVALID_ARG and "no device" in p.last_error()
    for ids, n in (([a, b], 384), ([a, b], 512), ([a, c], 128), ([a, b], 100), ([a], 640), ([a, b], 1 << 40), ([c, b], 256)):
        assert call(ids, n) == K.ERR_NOT_SHAREABLE, (ids, n)
    assert call([a, b], -128) == K.ERR_INVALID_ARG
    assert call([a, 7], 128) == K.ERR_BAD_REQUEST
    assert call([a], 0, layer=1) == K.ERR_INVALID_ARG
    assert p.L.kvpool_decode_attend_shared(None, 0, 0, None, 0, None, None, 0, None, None, None) == K.ERR_INVALID_ARG


@pytest.mark.parametrize("ts,hs,good", [
    (64, 64, False), (128, 64, False), (448, 64, False), (512, 64, True), (520, 64, True), (512, 72, False), (568, 72, True),
    (64, 64 * 99, False), (64, 64 * 100, True), (72, 72 * 99, False), (72, 72 * 99 + 64, True), (1 << 62, 64, True),
    (1 << 62, 1 << 62, False), (64, 1 << 62, True)])
def test_the_outer_axis_of_an_output_steps_over_the_inner_one(ts, hs, good):
    """8 heads of 100 tokens: a head of one token on a head of another is refused, however large both strides are."""
    o = heads(8, ts=ts, hs=hs)
    if not good:
        assert rope(T=100, q=heads(8), qo=o) == K.ERR_INVALID_ARG
        assert rope(T=100, k=heads(8), ko=o) == K.ERR_INVALID_ARG
    assert window([0], [0], [0], out=o, q_rows=100) == (K.OK if good else K.ERR_INVALID_ARG)
    assert window([0], [0], [0], out=o, q_rows=1) == K.OK
    assert window([0], [0], [0], out=heads(1, ts=ts, hs=0), q=heads(1), k=heads(1), v=heads(1)) == K.OK


def row(n, at, ts, hs, heads=None):
    """n heads of 64 bf16 values from value `at` of one buffer on."""
    return (P16 + 2 * at, ts, hs, n, 0)


def brute(a, na, b, nb, dim=64):
    pos = lambda x, n: {(x[0] - P16) // 2 + t * x[1] + h * x[2] + j for t in range(n) for h in range(x[3])  # noqa: E731
                        for j in range(dim)}
    return not pos(a, na).isdisjoint(pos(b, nb))


FUSED = [  # q, k (2 heads each unless said), output; the strides of each in one buffer
    (row(2, 0, 256, 64), row(2, 128, 256, 64), row(2, 0, 256, 64)),           # the queries' own place
    (row(2, 0, 256, 64), row(2, 128, 256, 64), row(2, 128, 256, 64)),         # the keys' place
    (row(2, 0, 256, 64), row(2, 128, 256, 64), row(2, 64, 256, 64)),          # a head behind the queries
    (row(2, 0, 256, 64), row(2, 128, 256, 64), row(2, 256, 256, 64)),         # a token behind them
    (row(2, 0, 384, 64), row(2, 128, 384, 64), row(2, 256, 384, 64)),         # a third part of the rows
    (row(2, 0, 384, 192), row(2, 64, 384, 192), row(2, 128, 384, 192)),       # parts of each head
    (row(2, 0, 384, 192), row(2, 64, 384, 192), row(2, 72, 384, 192)),
    (row(2, 0, 64, 64 * 20), row(2, 64 * 5, 64, 64 * 20), row(2, 64 * 10, 64, 64 * 20)),  # tokens inside heads
    (row(2, 0, 64, 64 * 20), row(2, 64 * 5, 64, 64 * 20), row(2, 64 * 8, 64, 64 * 20)),
    (row(2, 0, 0, 64), row(2, 128, 0, 64), row(2, 256, 128, 64)),             # one row for many
    (row(2, 0, 0, 64), row(2, 128, 0, 64), row(2, 128, 128, 64)),
    (row(2, 0, 384, 64), row(1, 128, 384, 0), row(2, 192, 384, 64)),          # one key head
    (row(2, 0, 384, 64), row(1, 128, 384, 0), row(2, 128, 384, 64)),
]


def meets(q, k, o, T):
    """Is that output neither the queries themselves nor apart from queries and keys?"""
    own = o[0] == q[0] and o[2] == q[2] and (T == 1 or o[1] == q[1])
    return not own and brute(o, T, q, T) or brute(o, T, k, T)


MET = [(i, T) for i in range(len(FUSED)) for T in (1, 2, 5) if meets(*FUSED[i], T)]


@pytest.mark.parametrize("case,T", MET)
def test_outputs_on_rows_that_are_read_are_refused(case, T):
    """(Those that are accepted are run in tests/test_gpu_rope.py.)"""
    q, k, o = FUSED[case]
    assert rope(T=T, q=q, k=k, qo=o, ko=row(k[3], 10 ** 6, 256, 64)) == K.ERR_INVALID_ARG
    if k[3] == q[3]:
        assert rope(T=T, q=k, k=q, qo=row(k[3], 10 ** 6, 256, 64), ko=o) == K.ERR_INVALID_ARG
    seg = ([T], [0], [T])
    a = K._WINDOW_ARGS.pack(K.BF16, 64, *q, *k, *k, *o, T, T, 0, 16, 0, 0.125, 0)
    seg = [np.array(x, np.int64) for x in seg]
    assert K.lib().kvpool_window_attend(a, 1, *(x.ctypes.data for x in seg), P16, 1 << 30, None) == K.ERR_INVALID_ARG


def test_outputs_on_each_other_are_refused():
    for at in (0, 64, 128 * 3 + 64):
        assert rope(T=4, q=row(2, 0, 128, 64), k=row(2, 4096, 128, 64), qo=row(2, 9000 * 8, 128, 64),
                    ko=row(2, 9000 * 8 + at, 128, 64)) == K.ERR_INVALID_ARG
    # strides that differ in one piece of memory
    assert rope(T=4, q=row(2, 0, 256, 64), qo=row(2, 128, 512, 64)) == K.ERR_INVALID_ARG


def test_share_bytes():
    from tests.test_abi_host import base_workload, cfg_of
    p = K.Pool(cfg_of(base_workload(layer_kinds=[K.HCA])))
    for n in (0, 1 << 50, -1):
        p.set_share_bytes(n)
    assert p.L.kvpool_set_share_bytes(None, 0) == K.ERR_INVALID_ARG
