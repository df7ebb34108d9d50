"""The kernels that read shared entries once, at any size: sharing is asked for where it would save little too, every
call is seen to have shared, and outputs are compared with the oracle and with the ordinary decode attention."""
import math

import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests import harness as H
from tests.gpu_harness import GpuCase, check_out
from tests.test_gpu_shared import BASE, TYPES, attend, build, close

pytestmark = pytest.mark.gpu
BF = (K.BF16, K.BF16)
ATTEND = K.KERNEL_NAMES.index("attend")


def launches(pool, call):
    """Attention kernels that the call launches."""
    pool.profile_enable(kinds=[], count=True)
    before = pool.profile_read(ATTEND)[1]
    call()
    n = pool.profile_read(ATTEND)[1] - before
    pool.profile_enable(False)
    return n


def shared(g, layer, slots, wids, top_k, n_shared, more=1):
    """attend() with sharing asked for: `more` attention kernels above those of the ordinary call."""
    q, qi = g.queries(layer, wids, 0)
    out = torch.empty((len(slots), g.HD), device="cuda")
    g.pool.set_share_bytes(0)
    n = launches(g.pool, lambda: g.pool.decode_attend_shared(layer, slots, n_shared, q, qi, top_k, out))
    assert n == launches(g.pool, lambda: g.pool.decode_attend(layer, slots, q, qi, top_k, out)) + more
    return attend(g, layer, slots, wids, top_k, n_shared)


def test_the_rule_decides_what_is_shared():
    g, _, slots = build(dict(BASE), 16, 128 * 1200, [i for i in range(16)], oracle=False)
    q, qi = g.queries(0, list(range(16)), 0)
    out = torch.empty((16, g.HD), device="cuda")
    call = lambda n: launches(g.pool, lambda: g.pool.decode_attend_shared(0, slots, n, q, qi, 0, out))  # noqa: E731
    assert (call(128 * 1200), call(128), call(0)) == (2, 1, 1)
    g.pool.set_share_bytes(0)
    assert (call(128 * 1200), call(128), call(0)) == (2, 2, 1)
    g.pool.set_share_bytes(1 << 50)
    assert call(128 * 1200) == 1
    g.pool.set_share_bytes(-1)
    assert (call(128 * 1200), call(128)) == (2, 1)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kind,heads,dim", [(K.HCA, 4, 64), (K.CSA_HCA, 2, 128), (K.HCA, 6, 128)])
def test_against_the_oracle(types, kind, heads, dim):
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], layer_kinds=[kind], heads=heads, head_dim=dim, idx_heads=1,
             idx_dim=32)
    g, o, slots = build(w, 5, 512, [0, 1, 130, 300, 5])
    # the same request twice, and in another order
    for pick in ([0, 1, 2, 3, 4], [3, 0, 3, 1]):
        ids = [slots[i] for i in pick]
        for n_shared in (512, 256, 128):
            out, ref = shared(g, 0, ids, pick, 16, n_shared)
            q, qi = H.queries(w, 0, pick, 0)
            rc, want, _ = o.decode_attend(0, ids, q, qi, 16)
            assert rc == 0
            check_out(out.cpu().numpy().reshape(want.shape), want, types[1])
            close(out, ref, *types[::-1])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("n,prefix", [(1, 128), (2, 128 * 33), (7, 128 * 65), (17, 128 * 200), (33, 128 * 31),
                                      (64, 128 * 129), (65, 128 * 64), (130, 128 * 40)])
def test_sizes_of_batch_and_prefix(n, prefix, types):
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=4, head_dim=128 if n % 2 else 64)
    g, _, slots = build(w, n, prefix, [(i * 37) % 300 for i in range(n)], oracle=False)
    out, ref = shared(g, 0, slots, list(range(n)), 0, prefix)
    close(out, ref, *types[::-1])


def test_more_requests_than_one_launch():
    w = dict(BASE, heads=4, head_dim=64)
    g, _, slots = build(w, 300, 256, [i % 3 for i in range(300)], oracle=False)
    out, ref = shared(g, 0, slots, list(range(300)), 0, 256, more=2)
    close(out, ref, *BF)


def scattered(w, n, blocks):
    """n requests behind one prefix whose blocks lie out of order: another request seals blocks in between, and half of the
    prefix is put into its place."""
    g = GpuCase(w, n + 2, 2 * blocks + 2 * n + 8, blocks + 4, n, 4)
    a, b = g.pool.alloc_request(), g.pool.alloc_request()
    for i in range(blocks // 2):
        g.append([a, b], [0, 1], [i * 128] * 2, [128, 128])
    g.pool.free_request(b)
    for i in range(blocks // 2, blocks):
        g.append([a], [0], [i * 128], [128])
    _, _, ids = g.pool.request_info(a)
    ids = [int(x) for x in ids]
    assert sum(y != x + 1 for x, y in zip(ids, ids[1:])) >= blocks - 3 and ids != sorted(ids)
    gk, gv, _ = g.tokens([0], [blocks * 128 - 128], [128])
    slots = [a]
    for i in range(1, n):
        slots.append(g.pool.alloc_request())
        g.pool.share_prefix(slots[-1], a, blocks * 128, gk, gv)
        g.append([slots[-1]], [i], [blocks * 128], [(i * 41) % 200 + 1])
    return g, slots


@pytest.mark.parametrize("types,heads,dim,n,blocks", [
    (BF, 4, 64, 3, 12), (BF, 4, 128, 20, 300), (BF, 4, 64, 50, 130), (BF, 4, 64, 34, 2060), (BF, 2, 128, 40, 2060),
    ((K.F32, K.F32), 4, 64, 5, 70), ((K.BF16, K.FP8_E4M3), 4, 128, 35, 70), ((K.F32, K.BF16), 4, 64, 4, 200)])
def test_scattered_blocks_and_a_request_twice(types, heads, dim, n, blocks):
    """Small products, products of 128 rows, FMAs, each through the block table, some requests named twice."""
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
    g, slots = scattered(w, n, blocks)
    pick = list(range(n))
    pick[n // 2], pick[-1] = 1, 0
    ids = [slots[i] for i in pick]
    out, ref = shared(g, 0, ids, pick, 0, blocks * 128)
    close(out, ref, *types[::-1])
    assert torch.equal(out[n // 2], out[1]) and torch.equal(out[-1], out[0])
    assert torch.equal(out, attend(g, 0, ids, pick, 0, blocks * 128)[0])  # the same bits again
    # a part of the prefix
    out, ref = shared(g, 0, ids, pick, 0, (blocks - 5) * 128)
    close(out, ref, *types[::-1])


def test_mixed_layers_and_offloaded_blocks():
    w = dict(BASE, n_layers=4, layer_kinds=[K.SWA_ONLY, K.CSA, K.HCA, K.CSA_HCA], heads=4, head_dim=64, csa_hot_slots=16,
             csa_host_slots=10)
    g, o, slots = build(w, 3, 1024, [40, 200, 3])
    g.pool.offload([int(b) for b in g.pool.request_info(slots[0])[2][:5]])
    for layer in range(4):
        out, ref = shared(g, layer, slots, [0, 1, 2], 32, 1024, more=layer >= 2)
        q, qi = H.queries(w, layer, [0, 1, 2], 0)
        rc, want, _ = o.decode_attend(layer, slots, q, qi, 32)
        check_out(out.cpu().numpy().reshape(want.shape), want, K.BF16)
        close(out, ref, *BF)


FORMS = [(BF, 4, 64, 9, 50), (BF, 4, 64, 40, 20), (BF, 4, 64, 40, 2050), ((K.F32, K.F32), 4, 64, 9, 50),
         ((K.BF16, K.FP8_E4M3), 4, 64, 9, 50)]


@pytest.mark.parametrize("types,heads,dim,n,entries", FORMS)
def test_graph_and_other_stream(types, heads, dim, n, entries):
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
    g, _, slots = build(w, n, 128 * entries, [i * 20 % 300 for i in range(n)], oracle=False)
    want, ref = shared(g, 0, slots, list(range(n)), 0, 128 * entries)
    close(want, ref, *types[::-1])
    q, qi = g.queries(0, list(range(n)), 0)
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


@pytest.mark.parametrize("types,heads,dim,n,entries", FORMS)
def test_one_request_does_not_reach_another(types, heads, dim, n, entries):
    """Queries of one request that are NaN, infinite or huge change nothing for the others of its tile."""
    w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
    g, _, slots = build(w, n, 128 * entries, [i * 20 % 300 for i in range(n)], oracle=False)
    want, _ = shared(g, 0, slots, list(range(n)), 0, 128 * entries)
    q, qi = g.queries(0, list(range(n)), 0)
    rest = [i for i in range(n) if i != 3]
    for x in (math.nan, math.inf, 1e4):
        bad = q.clone()
        bad[3] = q[3] * x if x == 1e4 else x
        out = torch.empty_like(want)
        g.pool.decode_attend_shared(0, slots, 128 * entries, bad, qi, 0, out)
        # (rescaling by warps may round the others' sums elsewhere)
        close(out[rest], want[rest], K.BF16, types[0])
        if x != 1e4:
            assert bool(torch.isnan(out[3]).all())
    assert g.pool.check_device() == 0


def test_large_scores():
    """Queries so large that one entry has all the weight: finite, and as the ordinary path."""
    for types, heads, dim, n, entries in FORMS[:4]:
        w = dict(BASE, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
        g, _, slots = build(w, n, 128 * entries, [i * 20 % 300 for i in range(n)], oracle=False)
        q, _ = g.queries(0, list(range(n)), 0)
        shared(g, 0, slots, list(range(n)), 0, 128 * entries)
        for scale in (300.0, 0.0):
            x = q * scale
            out, ref = torch.empty((n, g.HD), device="cuda"), torch.empty((n, g.HD), device="cuda")
            g.pool.decode_attend_shared(0, slots, 128 * entries, x, None, 0, out)
            g.pool.decode_attend(0, slots, x, None, 0, ref)
            assert bool(torch.isfinite(out).all())
            # scores of up to a few thousand are off by 2^-24 of themselves: 2^-10 in the weights
            assert float((out - ref).norm() / ref.norm()) <= 2.0 ** -8


def filled(w, n, entries, seed=1):
    """n requests behind a prefix whose HCA entries are random numbers (written into the pool as its layout says; the
    window's tokens are zeros), the entries and queries."""
    g = GpuCase(w, n, entries + 4, entries + 2, n, 4)
    slots = [g.pool.alloc_request() for _ in range(n)]
    step = 1 << 15
    z = torch.zeros((1, step, g.HD), dtype=g.tdtype, device="cuda")
    for p in range(0, 128 * entries, step):
        m = min(step, 128 * entries - p)
        zs = z[:, :m].contiguous()
        g.pool.append([slots[0]], [m], zs, zs, None)
    for s in slots[1:]:
        g.pool.share_prefix(s, slots[0], 128 * entries, z[:, :128].contiguous(), z[:, :128].contiguous())
    assert [int(x) for x in g.pool.request_info(slots[0])[2]] == list(range(entries))
    d = g.pool.layout(0)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kv = torch.randn((entries, 2, w["heads"], w["head_dim"]), device="cuda", generator=gen)
    kv = kv.to({K.F32: torch.float32, K.BF16: torch.bfloat16}[w["cache_dtype"]])
    pool = g.arena[d["hca_offset"]:d["hca_offset"] + entries * d["hca_block_bytes"]].view(entries, -1)
    pool[:, :2 * g.HD * g.vs] = kv.view(entries, -1).view(torch.uint8)
    return g, slots, kv, torch.randn((n, w["heads"], w["head_dim"]), device="cuda", generator=gen).to(g.tdtype)


def exact(kv, q):
    """In 64 bits, over the entries and a window of 128 zeros."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(q.shape[1]):
        s = q[:, h].double() @ kv[:, 0, h].double().T / math.sqrt(q.shape[2])
        m = s.amax(1, keepdim=True).clamp(min=0)
        p = torch.exp(s - m)
        out[:, h] = p @ kv[:, 1, h].double() / (p.sum(1, keepdim=True) + 128 * torch.exp(-m))
    return out


def off(w, n, entries):
    """The outputs' distance from 64 bits, of their norm."""
    g, slots, kv, q = filled(w, n, entries)
    g.pool.set_share_bytes(0)
    out = torch.empty(q.shape, device="cuda")
    assert launches(g.pool, lambda: g.pool.decode_attend_shared(0, slots, 128 * entries, q, None, 0, out)) == 2
    assert g.pool.check_device() == 0
    want = exact(kv, q)
    return float((out.double() - want).norm() / want.norm())


@pytest.mark.parametrize("heads,dim,n,entries", [(4, 64, 64, 8192), (4, 128, 64, 8192), (8, 128, 128, 8192)])
def test_more_runs_than_partials_have_places(heads, dim, n, entries):
    """Batches whose runs do not all get a place for their partials get as many as there are: runs stay short, and their
    sums (which the tensor core cuts off, tile after tile) within what close() allows."""
    assert off(dict(BASE, heads=heads, head_dim=dim), n, entries) <= 2.0 ** -18


def test_entries_are_not_shared_where_their_partials_would_be_too_many():
    """256 requests with 16 partials each of their windows and entries fill all places: the call is the ordinary one,
    which takes them, and not refused."""
    n, blocks = 256, 127
    w = dict(BASE, heads=4, head_dim=64, n_win=128 * blocks)
    g = GpuCase(w, n, blocks + 2, blocks + 2, n, 4)
    slots = [g.pool.alloc_request() for _ in range(n)]
    k, v, _ = g.tokens([0], [0], [128 * blocks])
    g.pool.append([slots[0]], [128 * blocks], k, v, None)
    for s in slots[1:]:
        g.pool.share_prefix(s, slots[0], 128 * blocks, k, v)
    out, ref = shared(g, 0, slots, list(range(n)), 0, 128 * blocks, more=0)
    assert torch.equal(out, ref)
    few, _ = shared(g, 0, slots[:9], list(range(9)), 0, 128 * blocks)  # fewer requests share
    close(few, ref[:9], *BF)


@pytest.mark.parametrize("heads,dim,n,entries", [(64, 64, 30, 16384), (64, 64, 16, 32768)])
def test_long_runs_of_the_small_products(heads, dim, n, entries):
    """8,192 and 16,384 entries to a CTA, whose sums the tensor core would cut off 1,536 times: still within close()."""
    assert off(dict(BASE, m=32, heads=heads, head_dim=dim), n, entries) <= 2.0 ** -18


@pytest.mark.parametrize("heads,dim,n,entries", [(64, 64, 256, 8192), (16, 128, 64, 16500), (8, 128, 128, 32768), (32, 128, 34, 9000),
                                                 (64, 64, 40, 16001)])
def test_long_runs_of_the_products_of_128_rows(heads, dim, n, entries):
    """Runs of 8 to 63 tiles, in sums of 8 that join: within close(), however long the run."""
    assert off(dict(BASE, m=32, heads=heads, head_dim=dim), n, entries) <= 2.0 ** -18


def test_growing_scores_in_long_runs():
    """Scores that grow along a run of 32 tiles, so that each of its sums outweighs those before it, and that fall, so that
    the last ones hardly count."""
    heads, dim, n, entries = 64, 64, 40, 8192
    g, slots, kv, q = filled(dict(BASE, heads=heads, head_dim=dim), n, entries)
    g.pool.set_share_bytes(0)
    d = g.pool.layout(0)
    pool = g.arena[d["hca_offset"]:d["hca_offset"] + entries * d["hca_block_bytes"]].view(entries, -1)
    q.fill_(1.0)
    for sign in (1, -1):
        kv[:, 0] = (sign * torch.arange(entries, device="cuda") / 1000)[:, None, None].bfloat16()  # scores up to 65
        pool[:, :2 * g.HD * 2] = kv.view(entries, -1).view(torch.uint8)
        out = torch.empty(q.shape, device="cuda")
        g.pool.decode_attend_shared(0, slots, 128 * entries, q, None, 0, out)
        assert g.pool.check_device() == 0
        want = exact(kv, q)
        # scores of 65 are off by at most 2 * 68 * 2^-24 * 65: 2^-10.9 in the worst weight, far less in their sum
        assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -13


@pytest.mark.parametrize("types,heads,dim,n,entries,pays", [
    # (steps as shared / each its own: the slower of the two takes 1.2 to 8 times as long)
    (BF, 16, 128, 64, 1024, True), (BF, 16, 128, 16, 128, False), (BF, 4, 64, 16, 4096, True),
    ((K.BF16, K.FP8_E4M3), 16, 128, 8, 8192, False), ((K.F32, K.FP8_E4M3), 16, 128, 4, 8192, False),
    ((K.BF16, K.FP8_E4M3), 16, 128, 32, 2048, False), ((K.BF16, K.FP8_E4M3), 4, 64, 64, 8192, True),
    ((K.F32, K.BF16), 16, 128, 8, 8192, False), ((K.F32, K.BF16), 16, 64, 64, 8192, True),
    ((K.F32, K.F32), 16, 128, 2, 4096, False), ((K.F32, K.F32), 16, 128, 64, 2048, True),
    ((K.BF16, K.F32), 16, 128, 32, 2048, True)])
def test_the_rule_takes_the_quicker_side(types, heads, dim, n, entries, pays):
    w = dict(BASE, m=32, in_dtype=types[0], cache_dtype=types[1], heads=heads, head_dim=dim)
    g = GpuCase(w, n, entries + 4, entries + 2, n, 4)
    slots = [g.pool.alloc_request() for _ in range(n)]
    z = torch.zeros((1, 128 * 128, g.HD), dtype=g.tdtype, device="cuda")
    for _ in range(entries // 128):
        g.pool.append([slots[0]], [128 * 128], z, z, None)
    for s in slots[1:]:
        g.pool.share_prefix(s, slots[0], 128 * entries, z[:, :128].contiguous(), z[:, :128].contiguous())
    q = torch.zeros((n, g.HD), dtype=g.tdtype, device="cuda")
    out = torch.empty((n, g.HD), device="cuda")
    assert launches(g.pool, lambda: g.pool.decode_attend_shared(0, slots, 128 * entries, q, None, 0, out)) == 1 + pays


def test_a_batch_too_large_for_the_ordinary_call_shares():
    n, entries = 256, 16400
    g, slots, kv, q = filled(dict(BASE, m=32, heads=4, head_dim=64), n, entries)
    out = torch.empty(q.shape, device="cuda")
    assert g.pool.decode_attend(0, slots, q, None, 0, out, check=False) == K.ERR_INVALID_ARG
    want = exact(kv, q)
    for nbytes in (-1, 1 << 50):
        g.pool.set_share_bytes(nbytes)
        out.zero_()
        g.pool.decode_attend_shared(0, slots, 128 * entries, q, None, 0, out)
        assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -18
