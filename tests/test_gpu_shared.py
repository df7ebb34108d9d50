"""Decode attention of a batch behind a shared prefix: against the oracle, and
against the ordinary decode attention of the same pool."""
import math

import numpy as np
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from heterogeneous_compressed_kv_gb300.gen import workloads as W
from tests import harness as H
from tests.gpu_harness import GpuCase, check_out

pytestmark = pytest.mark.gpu

BASE = dict(W.COMMON, name="shared", n_layers=1, layer_kinds=[K.HCA], heads=16, head_dim=128, idx_heads=4, idx_dim=64,
            in_dtype=K.BF16, cache_dtype=K.BF16, n_win=128, top_k=64, seed=11)


def build(w, n, prefix, own, oracle=True, first=None):
    """A pool (and the oracle) of n requests behind one prefix, request i with own[i] tokens of its own."""
    blocks = prefix // 128 + int(sum(x // 128 for x in own)) + 8
    mbpr = prefix // 128 + max(own) // 128 + 2
    g = GpuCase(w, n + 1, blocks, mbpr, max(n, 1), 4096)
    o = H.make_oracle(w, n + 1, blocks, mbpr) if oracle else None
    slots = [g.pool.alloc_request() for _ in range(n)]
    for s in slots:
        assert o is None or o.alloc_request() == (0, s)
    step = 2048
    for p0 in range(0, prefix, step):
        g.append([slots[0]], [0], [p0], [min(step, prefix - p0)])
    if o is not None:
        k, v, x = H.tokens(w, [0], [0], [prefix])
        assert o.append([slots[0]], [prefix], k, v, x) == 0
    wl = min(prefix, w["n_win"])
    gk, gv, _ = g.tokens([0], [prefix - wl], [wl])
    for s in slots[1:]:
        g.pool.share_prefix(s, slots[0], prefix, gk, gv)
        if o is not None:
            k, v, _ = H.tokens(w, [0], [prefix - wl], [wl])
            assert o.share_prefix(s, slots[0], prefix, k, v) == 0
    for i, s in enumerate(slots):
        if own[i]:
            g.append([s], [i], [prefix], [own[i]])
            if o is not None:
                k, v, x = H.tokens(w, [i], [prefix], [own[i]])
                assert o.append([s], [own[i]], k, v, x) == 0
    return g, o, slots


def attend(g, layer, slots, wids, top_k, n_shared, stream=None):
    q, qi = g.queries(layer, wids, 0)
    out = torch.full((len(slots), g.HD), math.nan, device="cuda")
    tk = torch.full((len(slots), max(top_k, 1)), -7, dtype=torch.int32, device="cuda")
    g.pool.decode_attend_shared(layer, slots, n_shared, q, qi, top_k, out, tk if top_k else None, stream=stream)
    ref = torch.empty_like(out)
    rk = torch.full_like(tk, -7)
    g.pool.decode_attend(layer, slots, q, qi, top_k, ref, rk if top_k else None, stream=stream)
    assert g.pool.check_device() == 0
    assert torch.equal(tk, rk)
    return out, ref


def close(out, ref, cache, in_dtype):
    """Both are fp32 sums of the same terms: each side's scores, weights and sums are off by a few 2^-24 of theirs (bounded
    by 2^-18 of the outputs' norm at scores of this size), except an fp8 cache's weights in the ordinary path, rounded to
    f16 (half a step, 2^-11 of each weight)."""
    rel = float((out.double() - ref.double()).norm() / ref.double().norm())
    assert rel <= (2.0 ** -11 if cache == K.FP8_E4M3 else 2.0 ** -18), rel


TYPES = [(K.F32, K.F32), (K.F32, K.BF16), (K.F32, K.FP8_E4M3), (K.BF16, K.F32), (K.BF16, K.BF16), (K.BF16, K.FP8_E4M3)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kind,heads,dim", [(K.HCA, 4, 64), (K.CSA_HCA, 2, 128), (K.HCA, 6, 128)])
def test_against_the_oracle(types, kind, heads, dim):
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], layer_kinds=[kind], heads=heads, head_dim=dim, idx_heads=1,
             idx_dim=32)
    g, o, slots = build(w, 5, 512, [0, 1, 130, 300, 5])
    wids = list(range(5))
    for n_shared in (512, 256, 128, 0):
        out, ref = attend(g, 0, slots, wids, 16, n_shared)
        q, qi = H.queries(w, 0, wids, 0)
        rc, want, _ = o.decode_attend(0, slots, q, qi, 16)
        assert rc == 0
        check_out(out.cpu().numpy().reshape(want.shape), want, types[1])
        close(out, ref, *types[::-1])


@pytest.mark.parametrize("types", [(K.BF16, K.BF16), (K.F32, K.F32), (K.BF16, K.FP8_E4M3), (K.F32, K.BF16)])
@pytest.mark.parametrize("n,prefix", [(1, 128), (2, 128 * 33), (7, 128 * 65), (17, 128 * 200), (33, 128 * 31),
                                      (64, 128 * 129), (65, 128 * 64), (130, 128 * 40)])
def test_sizes_of_batch_and_prefix(n, prefix, types):
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=4, head_dim=128 if n % 2 else 64)
    g, _, slots = build(w, n, prefix, [(i * 37) % 300 for i in range(n)], oracle=False)
    out, ref = attend(g, 0, slots, list(range(n)), 0, prefix)
    close(out, ref, *types[::-1])


@pytest.mark.parametrize("n,entries,heads,dim", [(33, 2048, 4, 64), (64, 2049, 2, 128), (129, 2300, 4, 64), (40, 2175, 16, 128)])
def test_many_entries_and_requests(n, entries, heads, dim):
    """Enough of both for the products of 128 rows: whole and ragged tiles, one and two of them, few and many splits."""
    w = dict(BASE, heads=heads, head_dim=dim)
    g, _, slots = build(w, n, 128 * entries, [(i * 37) % 200 for i in range(n)], oracle=False)
    out, ref = attend(g, 0, slots, list(range(n)), 0, 128 * entries)
    close(out, ref, K.BF16, K.BF16)
    assert torch.equal(out, attend(g, 0, slots, list(range(n)), 0, 128 * entries)[0])


def test_growing_scores_rescale_the_outputs():
    """Entries whose scores grow along the prefix, so that every row's maximum grows by more than a rescaling's step
    again and again."""
    w = dict(BASE, heads=4, head_dim=64)
    n, entries = 40, 2048
    blocks = entries + 8
    g = GpuCase(w, n, blocks, entries + 2, n, 4)
    slots = [g.pool.alloc_request() for _ in range(n)]
    q = torch.ones((n, g.HD), device="cuda", dtype=torch.bfloat16)
    for p0 in range(0, 128 * entries, 2048):
        t = torch.arange(p0, p0 + 2048, device="cuda", dtype=torch.float32)
        k = (t / 40000)[:, None].expand(2048, g.HD).to(torch.bfloat16).contiguous()  # scores up to 64 * 6.5 / 8 = 52
        v = torch.randn((2048, g.HD), device="cuda").to(torch.bfloat16)
        g.pool.append([slots[0]], [2048], k, v, None)
    for s in slots[1:]:
        g.pool.share_prefix(s, slots[0], 128 * entries, k[-128:].contiguous(), v[-128:].contiguous())
    out, ref = torch.empty((n, g.HD), device="cuda"), torch.empty((n, g.HD), device="cuda")
    g.pool.decode_attend_shared(0, slots, 128 * entries, q, None, 0, out)
    g.pool.decode_attend(0, slots, q, None, 0, ref)
    assert g.pool.check_device() == 0
    # scores of 52 are off by at most 2 * 68 * 2^-24 * 64 * 6.5 / 8: 2^-11 in the worst weight, far less in their sum
    assert float((out - ref).norm() / ref.norm()) <= 2.0 ** -13


def test_more_requests_than_one_launch():
    w = dict(BASE, heads=4, head_dim=64)
    g, _, slots = build(w, 300, 256, [i % 3 for i in range(300)], oracle=False)
    out, ref = attend(g, 0, slots, list(range(300)), 0, 256)
    close(out, ref, K.BF16, K.BF16)


def test_scattered_blocks_and_a_request_twice():
    """Prefix blocks out of order in memory (ids freed by others in between), the same request twice in a batch."""
    w = dict(BASE, heads=4, head_dim=64)
    g = GpuCase(w, 8, 64, 40, 8, 64)
    a, b, c = (g.pool.alloc_request() for _ in range(3))
    for i in range(6):  # a and b seal blocks in turn
        g.append([a, b], [0, 1], [i * 128] * 2, [128, 128])
    g.pool.free_request(b)
    for i in range(6, 12):  # a goes on in b's freed blocks
        g.append([a], [0], [i * 128], [128])
    _, _, ids = g.pool.request_info(a)
    assert any(int(y) != int(x) + 1 for x, y in zip(ids, ids[1:]))
    gk, gv, _ = g.tokens([0], [1536 - 128], [128])
    g.pool.share_prefix(c, a, 1536, gk, gv)
    g.append([c], [5], [1536], [77])
    slots = [a, c, c, a]
    out, ref = attend(g, 0, slots, [0, 1, 1, 2], 0, 1536)
    close(out, ref, K.BF16, K.BF16)
    assert torch.equal(out[1], out[2])
    assert torch.equal(out, attend(g, 0, slots, [0, 1, 1, 2], 0, 1536)[0])  # the same bits again


def test_mixed_layers_and_offloaded_blocks():
    w = dict(BASE, n_layers=4, layer_kinds=[K.SWA_ONLY, K.CSA, K.HCA, K.CSA_HCA], heads=4, head_dim=64, csa_hot_slots=16,
             csa_host_slots=10)
    g, o, slots = build(w, 3, 1024, [40, 200, 3])
    g.pool.offload([int(b) for b in g.pool.request_info(slots[0])[2][:5]])
    for layer in range(4):
        out, ref = attend(g, layer, slots, [0, 1, 2], 32, 1024)
        q, qi = H.queries(w, layer, [0, 1, 2], 0)
        rc, want, _ = o.decode_attend(layer, slots, q, qi, 32)
        check_out(out.cpu().numpy().reshape(want.shape), want, K.BF16)
        close(out, ref, K.BF16, K.BF16)


def test_large_scores():
    """Queries so large that one entry has all the weight: finite, and as the ordinary path."""
    w = dict(BASE, heads=4, head_dim=64, in_dtype=K.F32, cache_dtype=K.F32)
    g, _, slots = build(w, 3, 1280, [0, 9, 140], oracle=False)
    q, _ = g.queries(0, [0, 1, 2], 0)
    for scale in (300.0, 0.0):
        x = q * scale
        out, ref = torch.empty((3, g.HD), device="cuda"), torch.empty((3, g.HD), device="cuda")
        g.pool.decode_attend_shared(0, slots, 1280, x, None, 0, out)
        g.pool.decode_attend(0, slots, x, None, 0, ref)
        assert bool(torch.isfinite(out).all())
        # scores of up to a few thousand are off by 2^-24 of themselves: 2^-10 in the weights
        assert float((out - ref).norm() / ref.norm()) <= 2.0 ** -8


def test_graph_and_other_stream():
    w = dict(BASE, heads=4, head_dim=128)
    g, _, slots = build(w, 9, 128 * 50, [i * 20 for i in range(9)], oracle=False)
    q, qi = g.queries(0, list(range(9)), 0)
    want = torch.empty((9, g.HD), device="cuda")
    g.pool.decode_attend_shared(0, slots, 6400, q, qi, 0, want)
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), torch.zeros_like(want)
    g.pool.decode_attend_shared(0, slots, 6400, q, qi, 0, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.pool.decode_attend_shared(0, slots, 6400, q, qi, 0, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_layer_as_a_model_runs_it():
    """Norms and rotation, the prompt's window attention, the append, a shared prefix and a decode step together: the
    window layer's single-token output is the same from the cache as from the raw rows."""
    H_, D, Wn, n = 4, 64, 128, 256
    w = dict(BASE, n_layers=2, layer_kinds=[K.SWA_ONLY, K.HCA], heads=H_, head_dim=D)
    g = GpuCase(w, 4, 32, 16, 4, 16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((n + 2, 3 * H_, D), device="cuda", generator=gen).bfloat16()
    tab, pos = K.rope_table(D), torch.arange(n + 2, device="cuda")
    pos[n + 1] = n  # both requests' new token is at position n
    q, k = K.qk_norm_rope(rows[:, :H_], rows[:, H_:2 * H_], pos, tab)
    v = rows[:, 2 * H_:].contiguous()
    prompt = K.window_attend(q[:n], k[:n], v[:n], [n], [0], [n], Wn)
    assert bool(torch.isfinite(prompt).all())
    a, b = g.pool.alloc_request(), g.pool.alloc_request()
    two = lambda t: torch.stack([t, t])  # noqa: E731  (both layers keep the same rows)
    g.pool.append([a], [n], two(k[:n]), two(v[:n]), None)
    g.pool.share_prefix(b, a, n, two(k[n - Wn:n]), two(v[n - Wn:n]))
    g.pool.append([a, b], [1, 1], two(k[n:]), two(v[n:]), None)
    new = q[n:].contiguous()
    out = torch.empty((2, H_, D), device="cuda")
    g.pool.decode_attend_shared(0, [a, b], n, new, None, 0, out)
    ka, va = (torch.cat([x[:n], x[n:n + 1], x[:n], x[n + 1:]]) for x in (k, v))
    raw = K.window_attend(new, ka, va, [1, 1], [0, n + 1], [n + 1, n + 1], Wn)
    # raw rounds its weights and output to bf16: half a step each of the output's terms, here of order one
    assert float((raw.float() - out).norm() / out.norm()) <= 2.0 ** -7
    shared, plain = torch.empty_like(out), torch.empty_like(out)
    g.pool.decode_attend_shared(1, [a, b], n, new, None, 0, shared)
    g.pool.decode_attend(1, [a, b], new, None, 0, plain)
    assert g.pool.check_device() == 0
    close(shared, plain, K.BF16, K.BF16)


def size_of(w, n, prefix):
    size = {K.F32: 4, K.BF16: 2, K.FP8_E4M3: 1}[w["cache_dtype"]]
    return (n - 1) * (prefix // 128) * 2 * w["heads"] * w["head_dim"] * size


@pytest.mark.parametrize("types,heads,dim,n,entries", [
    # bf16 on the small products: 16, 32 and 64 requests to a CTA, whole and ragged stages, one CTA's requests and more
    ((K.BF16, K.BF16), 16, 128, 2, 8200), ((K.BF16, K.BF16), 16, 128, 9, 1101), ((K.BF16, K.BF16), 16, 128, 17, 600),
    ((K.BF16, K.BF16), 16, 64, 31, 577), ((K.BF16, K.BF16), 16, 128, 33, 257), ((K.BF16, K.BF16), 16, 128, 65, 129),
    ((K.BF16, K.BF16), 16, 64, 150, 113),
    # the products of 128 rows
    ((K.BF16, K.BF16), 16, 128, 34, 2050), ((K.BF16, K.BF16), 4, 128, 130, 2100), ((K.BF16, K.BF16), 16, 64, 40, 2309),
    # FMAs
    ((K.F32, K.F32), 16, 128, 5, 1025), ((K.F32, K.F32), 4, 64, 33, 1101), ((K.BF16, K.FP8_E4M3), 16, 128, 33, 515),
    ((K.F32, K.BF16), 16, 64, 64, 300), ((K.BF16, K.F32), 4, 128, 50, 400), ((K.F32, K.FP8_E4M3), 16, 64, 70, 500)])
def test_sizes_that_share(types, heads, dim, n, entries):
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
    assert size_of(w, n, 128 * entries) >= 64 << 20
    g, _, slots = build(w, n, 128 * entries, [(i * 37) % 300 for i in range(n)], oracle=False)
    out, ref = attend(g, 0, slots, list(range(n)), 0, 128 * entries)
    close(out, ref, *types[::-1])
    assert torch.equal(out, attend(g, 0, slots, list(range(n)), 0, 128 * entries)[0])  # the same bits again
    # a shorter prefix of the same requests (some of it then each request's own), and one too short to share
    for blocks in (entries - 1, 3):
        out, ref = attend(g, 0, slots, list(range(n)), 0, 128 * blocks)
        close(out, ref, *types[::-1])


@pytest.mark.parametrize("dim,n,entries", [(128, 9, 1200), (64, 40, 2100)])
def test_layers_with_csa_share_beside_the_select(dim, n, entries):
    """The shared entries' kernel on the stream beside the indexer's select, before and behind the [HCA | window] part."""
    w = dict(BASE, layer_kinds=[K.CSA_HCA], heads=16, head_dim=dim, idx_heads=1, idx_dim=32)
    assert size_of(w, n, 128 * entries) >= 64 << 20
    g, _, slots = build(w, n, 128 * entries, [i * 9 for i in range(n)], oracle=False)
    for top_k in (16, 0):
        out, ref = attend(g, 0, slots, list(range(n)), top_k, 128 * entries)
        close(out, ref, K.BF16, K.BF16)


def test_more_requests_than_one_launch_share():
    w = dict(BASE, heads=4, head_dim=64)
    g, _, slots = build(w, 300, 128 * 300, [i % 3 for i in range(300)], oracle=False)
    assert size_of(w, 300, 128 * 300) >= 64 << 20
    out, ref = attend(g, 0, slots, list(range(300)), 0, 128 * 300)
    close(out, ref, K.BF16, K.BF16)


@pytest.mark.parametrize("n,entries", [(9, 1200), (40, 2100)])
def test_graph_and_other_stream_where_entries_are_shared(n, entries):
    w = dict(BASE, heads=16, head_dim=128)
    g, _, slots = build(w, n, 128 * entries, [i * 20 for i in range(n)], oracle=False)
    q, qi = g.queries(0, list(range(n)), 0)
    want = torch.empty((n, g.HD), device="cuda")
    g.pool.decode_attend_shared(0, slots, 128 * entries, q, qi, 0, want)
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), torch.zeros_like(want)
    g.pool.decode_attend_shared(0, slots, 128 * entries, q, qi, 0, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):  # each behind the one before, in the same partials
            g.pool.decode_attend_shared(0, slots, 128 * entries, q, qi, 0, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and g.pool.check_device() == 0


def test_large_scores_where_entries_are_shared():
    """Queries so large that one entry has all the weight, and queries of zeros."""
    for types, heads, dim, n, entries in (((K.BF16, K.BF16), 16, 128, 9, 1100), ((K.BF16, K.BF16), 16, 64, 40, 2048),
                                          ((K.F32, K.F32), 4, 64, 33, 1100)):
        w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
        g, _, slots = build(w, n, 128 * entries, [i * 3 for i in range(n)], oracle=False)
        q, _ = g.queries(0, list(range(n)), 0)
        for scale in (300.0, 0.0):
            x = q * scale
            out, ref = torch.empty((n, g.HD), device="cuda"), torch.empty((n, g.HD), device="cuda")
            g.pool.decode_attend_shared(0, slots, 128 * entries, x, None, 0, out)
            g.pool.decode_attend(0, slots, x, None, 0, ref)
            assert bool(torch.isfinite(out).all())
            # scores of up to a few thousand are off by 2^-24 of themselves: 2^-10 in the weights
            assert float((out - ref).norm() / ref.norm()) <= 2.0 ** -8
