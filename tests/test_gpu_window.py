"""Window attention with first tokens that stay visible against the formula in
64 bits."""
import math

import numpy as np
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def no_wait_runs_out():
    yield
    assert K.window_check() == (K.OK, 0)


def formula(q, k, v, ql, ks, kl, window, sink, scale):
    """(out, lse, mass) in 64 bits: mass = sum of p |v|, which the tolerances count in."""
    q, k, v = q.double(), k.double(), v.double()
    group = q.shape[1] // k.shape[1]
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    at = 0
    for n, k0, m in zip(ql, ks, kl):
        p = torch.arange(m - n, m, device=q.device)[:, None]
        t = torch.arange(m, device=q.device)[None]
        see = (t <= p) & ((t > p - window) | (t < sink))
        kk, vv = (x[k0:k0 + m].repeat_interleave(group, 1) for x in (k, v))
        s = torch.einsum("nhd,mhd->hnm", q[at:at + n], kk) * scale
        s = torch.where(see, s, -math.inf)
        z = torch.logsumexp(s, -1, keepdim=True)
        w = torch.where(see, torch.exp(s - torch.where(z == -math.inf, 0.0, z)), 0.0)
        vv = torch.where(see.any(0)[:, None, None], vv, 0.0)
        out[at:at + n] = torch.einsum("hnm,mhd->nhd", w, vv)
        mass[at:at + n] = torch.einsum("hnm,mhd->nhd", w, vv.abs())
        lse[at:at + n] = z[..., 0].T if m else -math.inf
        at += n
    return out, lse, mass


def check(got, lse, want, q, k, scale, dtype, n_keys):
    ref, z, mass = want
    # a score's sum of D products in fp32 is off by at most D 2^-24 |q||k|, twice for products and order; a weight by
    # that, by 2^-20 (its exponential and the rescaling) and by the sum over the keys; with bf16 each weight is rounded
    # once more (half a step), and the output too
    fin = torch.finfo(dtype).eps / 2
    qk = scale * float(q.double().norm(dim=-1).max() * k.double().nan_to_num(0, 0, 0).norm(dim=-1).max())
    s_err = 2 * (q.shape[-1] + 4) * 2.0 ** -24 * qk
    rel = 2 * s_err + 2.0 ** -20 + n_keys * 2.0 ** -24
    tol = fin * ref.abs() + (rel + (fin if dtype == BF else 0)) * mass * 1.01 + 1e-30
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if lse is not None:
        dead = z == -math.inf
        assert torch.equal(dead, lse == -math.inf)
        e = (lse.double() - z)[~dead].abs()
        tol = (rel + 2.0 ** -23 * z.abs())[~dead]
        assert bool((e <= tol).all()), float((e / tol).max())


def inputs(ql, kl, hq, hk, d, dtype, seed=0, gap=0):
    """Rows of all segments, `gap` rows of NaN between their cached tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((int(sum(ql)), hq, d), device="cuda", generator=g).to(dtype)
    ks, rows = [], gap
    for m in kl:
        ks.append(rows)
        rows += m + gap
    k, v = (torch.full((rows, hk, d), math.nan, device="cuda", dtype=dtype) for _ in range(2))
    for k0, m in zip(ks, kl):
        k[k0:k0 + m] = torch.randn((m, hk, d), device="cuda", generator=g).to(dtype)
        v[k0:k0 + m] = torch.randn((m, hk, d), device="cuda", generator=g).to(dtype)
    return q, k, v, ks


def run(ql, kl, hq, hk, d, dtype, window, sink, seed=0, gap=3):
    q, k, v, ks = inputs(ql, kl, hq, hk, d, dtype, seed, gap)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = K.window_attend(q, k, v, ql, ks, kl, window, sink, lse=lse)
    scale = 1 / math.sqrt(d)
    check(out, lse, formula(q, k, v, ql, ks, kl, window, sink, scale), q, k, scale, dtype, max(max(kl), 1))


SHAPES = [  # q_len, k_len, window, sinks
    ([1], [1], 1, 0), ([1], [1], 0, 0), ([1], [1], 0, 1), ([2], [2], 1, 0), ([5], [5], 16, 2),
    ([1, 1, 1], [1, 77, 300], 64, 4), ([1] * 9, [1, 2, 31, 32, 33, 127, 128, 129, 1000], 128, 0),
    ([64], [64], 64, 0), ([65], [200], 33, 3), ([130], [130], 1000, 0), ([127, 128, 129], [127, 128, 129], 128, 1),
    ([300], [1000], 128, 130), ([257, 1, 0, 40], [700, 513, 9, 40], 100, 5), ([10], [4], 8, 2), ([3], [0], 4, 4),
    ([0, 6], [5, 6], 4, 0), ([513], [2000], 256, 64), ([17], [4000], 3000, 1), ([200], [260], 0, 7), ([40], [40], 2 ** 31 - 1, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_formula(shape, d, dtype):
    ql, kl, window, sink = shape
    run(ql, kl, 4, 2, d, dtype, window, sink, seed=len(ql) + sum(kl))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (6, 2), (5, 1), (8, 1), (14, 2), (16, 1)])
@pytest.mark.parametrize("ql,kl", [([1, 1], [90, 700]), ([5, 2], [5, 640]), ([150], [400])])
def test_groups(ql, kl, hq, hk, dtype):
    run(ql, kl, hq, hk, 64, dtype, 100, 3, seed=hq)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_segments(dtype):
    r = np.random.RandomState(0)
    kl = r.randint(0, 90, 600).tolist()
    ql = [int(min(m, x)) for m, x in zip(kl, r.randint(0, 4, 600))]
    run(ql, kl, 2, 1, 64, dtype, 20, 2, gap=1)


@pytest.mark.parametrize("d", [64, 128])
def test_many_tiles_per_cta(d):
    """Prompts of more tiles than the GPU has multiprocessors: every CTA takes several, of different lengths."""
    run([1664, 1500, 700], [1664, 1800, 700], 16, 16, d, BF, 128, 4)
    run([4096], [4300], 16, 8, d, BF, 1000, 4)


def test_long_single_tokens_split_and_merge():
    run([1], [70001], 4, 1, 128, BF, 1 << 20, 0)
    run([1, 1], [20000, 5], 2, 2, 64, F32, 1 << 20, 0)
    run([2], [9000], 4, 4, 128, BF, 4096, 500)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("ql,kl,window,sink", [([200], [1000], 100, 4), ([1, 300], [900, 2000], 130, 140), ([17], [600], 64, 1),
                                               ([700], [5000], 256, 16)])
def test_rows_that_nobody_sees_may_hold_anything(ql, kl, window, sink, dtype):
    """NaN between the first tokens and the first query's window (tokens that were dropped there) changes nothing."""
    q, k, v, ks = inputs(ql, kl, 4, 2, 128, dtype, gap=1)
    want = K.window_attend(q, k, v, ql, ks, kl, window, sink)
    for n, k0, m in zip(ql, ks, kl):
        k[k0 + sink:k0 + m - n - window + 1] = math.nan
        v[k0 + sink:k0 + m - n - window + 1] = math.nan
    got = K.window_attend(q, k, v, ql, ks, kl, window, sink)
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30])
@pytest.mark.parametrize("ql", [[1], [40]])
def test_any_scale(ql, scale):
    q, k, v, ks = inputs(ql, [300], 4, 2, 64, BF)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = K.window_attend(q, k, v, ql, ks, [300], 100, 3, scale=scale, lse=lse)
    check(out, lse, formula(q, k, v, ql, ks, [300], 100, 3, scale), q, k, abs(scale), BF, 300)


@pytest.mark.parametrize("ql", [[1], [40]])
def test_broadcast_key_heads(ql):
    """One key head's rows seen as four by a stride of zero."""
    q, k, v, ks = inputs(ql, [300], 4, 1, 64, BF)
    want = K.window_attend(q, k, v, ql, ks, [300], 100, 3)
    got = K.window_attend(q, k.expand(-1, 4, -1), v.expand(-1, 4, -1), ql, ks, [300], 100, 3)
    # the same scores; weights are rounded to bf16 (half a step each) in either or both, and the outputs
    assert float((got.float() - want.float()).norm() / want.float().norm()) <= 2.0 ** -7


def test_two_streams_at_once():
    q, k, v, ks = inputs([300, 1], [900, 4000], 8, 2, 128, BF, gap=0)
    args = (q, k, v, [300, 1], ks, [900, 4000], 500, 4)
    want = K.window_attend(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(10):
        for s in streams:
            outs.append(K.window_attend(*args, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_large_scores_keep_the_softmax_finite():
    q, k, v, ks = inputs([40], [40], 2, 2, 64, BF)
    q, k = q * 40, k * 40  # scores in the thousands: one key has all the weight
    out = K.window_attend(q, k, v, [40], ks, [40], 16)
    want = formula(q, k, v, [40], ks, [40], 16, 0, 0.125)
    assert bool(torch.isfinite(out).all())
    near = (out.double() - want[0]).abs() <= 2.0 ** -6 * want[2] + 1e-6
    assert float(near.double().mean()) > 0.999  # ties between two keys within a score's rounding may fall either way


def test_views_other_rows_and_scale():
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.randn((300, 8 + 2 * 2, 64), device="cuda", generator=g).to(BF)
    q, k, v = rows[:, :8], rows[:, 8:10], rows[:, 10:]
    out = torch.full((310, 8, 64), 3.0, device="cuda", dtype=BF)
    got = K.window_attend(q[40:200], k, v, [100], [50], [180], 70, 2, scale=0.3, out=out[:160])
    assert got.data_ptr() == out.data_ptr()
    want = formula(q[40:140], k, v, [100], [50], [180], 70, 2, 0.3)
    check(got[:100], None, want, q, k, 0.3, BF, 180)
    assert bool((out[100:] == 3.0).all())  # rows behind the last segment
    # heads outermost
    kt = torch.randn((2, 300, 64), device="cuda", generator=g).to(BF).transpose(0, 1)
    got = K.window_attend(q, kt, v, [300], [0], [300], 64)
    check(got, None, formula(q, kt, v, [300], [0], [300], 64, 0, 0.125), q, kt, 0.125, BF, 300)


def test_overlapping_segments_read_the_same_rows():
    # two requests over one shared prompt's rows
    q, k, v, _ = inputs([3, 50], [100], 2, 1, 128, BF, gap=0)
    out = K.window_attend(q, k, v, [3, 50], [0, 10], [100, 90], 33, 1)
    scale = 1 / math.sqrt(128)
    check(out, None, formula(q, k, v, [3, 50], [0, 10], [100, 90], 33, 1, scale), q, k, scale, BF, 100)


@pytest.mark.parametrize("ql,kl", [([1, 1], [5000, 300]), ([400], [900])])
def test_same_bits_again_streams_and_graphs(ql, kl):
    q, k, v, ks = inputs(ql, kl, 4, 2, 128, BF, gap=0)
    args = (q, k, v, ql, ks, kl, 2048, 4)
    want = K.window_attend(*args)
    assert torch.equal(want, K.window_attend(*args))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = K.window_attend(*args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = [torch.empty(max(K.window_workspace(*args), 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], []
    for o, w in zip(outs, ws):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            K.window_attend(*args, out=o, workspace=w)
    q.mul_(-0.5)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    want = K.window_attend(*args)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_refusals():
    q, k, v, ks = inputs([4], [10], 4, 2, 64, BF, gap=0)
    ok = dict(q=q, k=k, v=v, q_len=[4], k_start=[0], k_len=[10], window=4)
    K.window_attend(**ok)
    for bad in (dict(q=q.half()), dict(k=k.float()), dict(v=v[:5]), dict(q=q.cpu()), dict(out=q[:3]),
                dict(out=q[:1].expand(4, 4, 64)), dict(lse=torch.empty((4, 4), device="cuda", dtype=BF)),
                dict(q_len=[4, 1]), dict(q_len=[1.5]), dict(k_start=[2 ** 70]), dict(q=q[..., :32])):
        with pytest.raises((ValueError, OverflowError)):
            K.window_attend(**{**ok, **bad})
    for bad in (dict(q_len=[5]), dict(k_len=[11]), dict(k_start=[1]), dict(window=-1), dict(n_sink=-1),
                dict(scale=math.inf)):
        with pytest.raises(K.KvpoolError):
            K.window_attend(**{**ok, **bad})
    qs, kss, vs, st = inputs([1], [3000], 4, 2, 64, BF, gap=0)
    call = dict(q=qs, k=kss, v=vs, q_len=[1], k_start=st, k_len=[3000], window=3000)
    if K.window_workspace(**call):
        with pytest.raises(K.KvpoolError):
            K.window_attend(**call, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("ql,kl,sink", [([150], [400], 7), ([150], [160], 40), ([200, 3], [200, 300], 0), ([20], [20], 9)])
def test_a_window_of_nothing_reads_the_first_tokens_alone(ql, kl, sink, dtype):
    """With window 0 no query sees a row behind the first tokens: NaN there changes nothing."""
    q, k, v, ks = inputs(ql, kl, 4, 2, 64, dtype, gap=1)
    want = formula(q, k, v, ql, ks, kl, 0, sink, 0.125)
    for k0, m in zip(ks, kl):
        k[k0 + sink:k0 + m] = math.nan
        v[k0 + sink:k0 + m] = math.nan
    lse = torch.empty(q.shape[:2], device="cuda")
    check(K.window_attend(q, k, v, ql, ks, kl, 0, sink, lse=lse), lse, want, q, k, 0.125, dtype, max(sink, 1))


def test_more_items_than_a_cta_works_out_at_its_start():
    """16,384 work items: over 96 for each of 152 persistent CTAs."""
    r = np.random.RandomState(2)
    ql = [int(x) for x in r.randint(17, 21, 256)]
    kl = [n + int(x) for n, x in zip(ql, r.randint(0, 30, 256))]
    run(ql, kl, 64, 64, 64, BF, 24, 2, gap=0)


@pytest.mark.parametrize("scale", [None, -0.3])
def test_workspace_of_the_same_arguments_is_enough(scale):
    """Scales that are not positive go to another form of the kernel, which may want another workspace."""
    q, k, v, ks = inputs([40], [5000], 2, 1, 64, BF)
    args = (q, k, v, [40], ks, [5000], 4096, 3)
    space = torch.empty(max(K.window_workspace(*args, scale=scale), 1), dtype=torch.uint8, device="cuda")
    assert space.numel() > 1
    got = K.window_attend(*args, scale=scale, workspace=space)
    s = 0.125 if scale is None else scale
    check(got, None, formula(q, k, v, [40], ks, [5000], 4096, 3, s), q, k, abs(s), BF, 5000)


def test_window_workspace_of_broadcast_queries():
    q = torch.zeros((1, 2, 64), device="cuda", dtype=BF).expand(40, -1, -1)
    k = torch.zeros((5000, 1, 64), device="cuda", dtype=BF)
    args = (q, k, k, [40], [0], [5000], 4096)
    assert K.window_workspace(*args) > 0
    assert K.window_attend(*args).shape == (40, 2, 64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(4, 4), (16, 2), (16, 1)])
@pytest.mark.parametrize("ql,kl,window,sink", [([1] * 6, [1, 40, 129, 1000, 4000, 9000], 4096, 4), ([1, 1], [8, 700], 128, 0),
                                               ([1], [70001], 1 << 20, 1)])
def test_single_tokens_hold_their_weights_in_16_bits(ql, kl, window, sink, hq, hk, d):
    """The output's own rounding is the one that shows: no half step of bf16 for the weights, whose two pieces leave
    2^-18 of each (half a step of half a step)."""
    q, k, v, ks = inputs(ql, kl, hq, hk, d, BF, seed=len(kl))
    q = q / 8  # many keys count, and the scores' own error stays small
    out = K.window_attend(q, k, v, ql, ks, kl, window, sink)
    scale = 1 / math.sqrt(d)
    ref, _, mass = formula(q, k, v, ql, ks, kl, window, sink, scale)
    qk = scale * float(q.double().norm(dim=-1).max() * k.double().nan_to_num(0, 0, 0).norm(dim=-1).max())
    n_keys = min(window + sink, max(kl))
    # as in check(), but a weight's rounding is 2^-18 (twice: in a sum of two products)
    rel = 4 * (d + 4) * 2.0 ** -24 * qk + 2.0 ** -20 + n_keys * 2.0 ** -24 + 2.0 ** -17
    tol = torch.finfo(BF).eps / 2 * ref.abs() + rel * mass * 1.01 + 1e-30
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


FORMS = [  # q_len, k_len, window, dtype, scale: single tokens, prompts (tensor cores, FMAs), keys split over CTAs
    ([1, 1], [40, 300], 64, BF, None), ([1, 1], [40, 300], 64, F32, None), ([1], [9000], 8000, BF, None),
    ([2], [9000], 8000, F32, None), ([60, 200], [60, 500], 128, BF, None), ([150], [5000], 4096, BF, None),
    ([60, 200], [60, 500], 128, F32, None), ([60, 200], [60, 500], 128, BF, -0.125), ([40], [5000], 4096, F32, None)]


@pytest.mark.parametrize("ql,kl,window,dtype,scale", FORMS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_score_that_is_not_finite_reaches_what_sees_it_and_nothing_else(ql, kl, window, dtype, scale, bad):
    """A NaN or an overflow among a query's own scores is no row that sees nothing: its outputs and its log-sum-exp are
    NaN.  A NaN among the values leaves the log-sum-exp alone."""
    q, k, v, ks = inputs(ql, kl, 4, 2, 64, dtype)
    s = 0.125 if scale is None else scale
    t = kl[-1] - ql[-1]  # the last segment's first query's own token, under key head 1
    want = formula(q, k, v, ql, ks, kl, window, 0, s)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    at = sum(ql[:-1])
    hit[at:at + min(window, ql[-1]), 2:] = True
    bad_k = k.clone()
    bad_k[ks[-1] + t, 1] = bad
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = K.window_attend(q, bad_k, v, ql, ks, kl, window, scale=scale, lse=lse)
    # (products of an infinity with queries of both signs sum to NaN)
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    other = [torch.where(hit[..., None] if x.dim() == 3 else hit, y, x) for x, y in
             ((out, want[0].to(dtype)), (lse, want[1].float()))]
    check(*other, want, q, k, abs(s), dtype, max(kl))
    bad_v = v.clone()
    bad_v[ks[-1] + t, 1, 5] = bad
    lse2 = torch.full(q.shape[:2], 7.0, device="cuda")
    out = K.window_attend(q, k, bad_v, ql, ks, kl, window, scale=scale, lse=lse2)
    check(out.nan_to_num(0, 0, 0) * 0, lse2, (want[0] * 0, want[1], want[2]), q, k, abs(s), dtype, max(kl))
    assert not bool(torch.isfinite(out[hit][:, 5]).any())


def test_scores_of_minus_infinity_alone():
    for ql, dtype in (([1], BF), ([1], F32), ([40], BF), ([40], F32)):
        q, k, v, ks = inputs(ql, [200], 2, 1, 64, dtype)
        q, k = q.abs() + 1, -torch.full_like(k, math.inf)
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = K.window_attend(q, k, v, ql, ks, [200], 64, 1, lse=lse)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
