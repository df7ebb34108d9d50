"""The 4-bit paged cache against its format and formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests import kv4_format as F

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, g, size=1.0):
    return (size * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def make(lens, page, hk, d, seed=0, ks=1.0, vs=1.0, spare=2, fill=0xFF):
    """A cache with a table for lens tokens (pages in no order, `fill` in every byte: NaN scales)."""
    r = np.random.RandomState(seed)
    need = [max(1, -(-n // page)) for n in lens]
    total = sum(need) + spare
    ids = r.permutation(total)
    table = torch.zeros((len(lens), max(need, default=1)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.from_numpy(ids[at:at + n].astype(np.int32))
        at += n
    pages = torch.full((total, K.kv4_page_bytes(hk, d, page)), fill, dtype=torch.uint8, device="cuda")
    return K.Kv4Cache(pages, hk, d, page, ks, vs), table.cuda()


def same(got, want):
    """Equal values, NaN for NaN."""
    got, want = got.double().cpu(), want.double().cpu()
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


def ok():
    assert K.window_check() == (K.OK, 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,hk,start,n_new", [
    (16, 1, [0], [1]), (16, 3, [5], [1]), (64, 2, [0, 7, 16], [33, 1, 0]), (128, 4, [1, 31, 100], [2, 200, 77]),
    (256, 1, [15, 16, 17, 0], [1, 1, 1, 16]), (1024, 2, [1000], [100]), (32, 16, [3] * 40, [1] * 40)])
def test_store_and_load(page, hk, start, n_new, d, dtype):
    g = gen(page + hk + d)
    cache, table = make([a + n + 20 for a, n in zip(start, n_new)], page, hk, d, ks=0.5, vs=4.0)
    n = sum(n_new)
    k, v = randn((n, hk, d), dtype, g), randn((n, hk, d), dtype, g, 7.0)
    cache.store(k, v, table, start, n_new)
    k2, v2 = cache.load(table, start, n_new, dtype=dtype)
    assert k2.dtype is dtype and same(k2, F.held(k, 0.5)) and same(v2, F.held(v, 4.0))
    ok()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_a_store_leaves_its_neighbours(d, page):
    """One token at a time over and between others: each place holds the last token stored there."""
    g, T, hk = gen(3), 70, 2
    cache, table = make([T], page, hk, d)
    k, v = randn((T, hk, d), BF, g), randn((T, hk, d), BF, g)
    cache.store(k, v, table, [0], [T])
    pages = cache.pages.clone()
    for t in (0, 1, 15, 16, 33, 34, 69):
        k[t], v[t] = randn((hk, d), BF, g, 3.0), randn((hk, d), BF, g, 3.0)
        cache.store(k[t:t + 1], v[t:t + 1], table, [t], [1])
    k2, v2 = cache.load(table, [0], [T])
    assert same(k2, F.held(k)) and same(v2, F.held(v))
    used = set(table.flatten().tolist())
    for i in range(pages.shape[0]):  # pages that are in no row stay as they were
        if i not in used:
            assert torch.equal(pages[i], cache.pages[i])
    ok()


def test_borders_and_special_values():
    """Values on the borders between codes, zeros, groups that a scale cannot hold, infinities and NaN."""
    d, rows = 128, []
    for s in (1.0, 0.4375, 2.0 ** -9, 288.0):  # scales that e4m3 has: the largest value 6 s keeps them
        x = torch.zeros(d)
        for i, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
            x[2 * i], x[2 * i + 1] = b * s, -b * s
        x[14] = 6 * s
        for grp in range(1, 8):
            x[16 * grp:16 * grp + 16] = x[:16] * (1 + (grp - 4) * 2.0 ** -7)
        rows.append(x)
    x = torch.zeros(d)
    x[16:32], x[32:48], x[48:64] = 1e5, 6 * 2.0 ** -10, 6.1 * 2.0 ** -10
    x[64], x[80], x[96], x[112] = math.inf, -math.inf, math.nan, 1e-40
    rows.append(x)
    x = torch.stack(rows)[:, None]
    for dtype in (F32, BF):
        y = x.to(dtype).cuda()
        cache, table = make([8], 16, 1, d)
        cache.store(y, y, table, [1], [5])
        k, v = cache.load(table, [1], [5], dtype=F32)
        assert same(k, F.held(y)) and same(v, F.held(y))
    ok()


def test_rows_of_a_fused_projection_and_given_outputs():
    g, T, hk, d = gen(5), 50, 2, 64
    rows = randn((T, 8, d), BF, g)
    k, v = rows[:, 4:6], rows[:, 6:8]
    cache, table = make([T], 32, hk, d)
    cache.store(k, v, table, [0], [T])
    both = torch.full((T + 3, 5, d), 9.0, dtype=F32, device="cuda")
    out = cache.load(table, [0], [T], out_k=both[:, 1:3], out_v=both[:, 3:])
    assert out[0].data_ptr() == both[:, 1:3].data_ptr()
    assert same(both[:T, 1:3], F.held(k)) and same(both[:T, 3:], F.held(v))
    assert bool((both[:, 0] == 9).all()) and bool((both[T:] == 9).all())
    with pytest.raises(K.KvpoolError):
        cache.load(table, [0], [T], out_k=both[:, 1:3], out_v=both[:, 2:4])
    ok()


# ---- attention ----------------------------------------------------------------


def fill(cache, table, lens, dtype, g, k_size=1.0, v_size=1.0):
    """Random tokens in the cache; what it holds of them, on the CPU."""
    hk, d = cache.kv_heads, cache.head_dim
    n = sum(lens)
    k = randn((n, hk, d), dtype, g, k_size)
    k *= torch.exp(0.5 * torch.randn((hk, d), device="cuda", generator=g)).to(dtype)
    v = randn((n, hk, d), dtype, g, v_size)
    cache.store(k, v, table, [0] * len(lens), lens)
    return F.held(k, cache.k_scale), F.held(v, cache.v_scale)


def check(q, k, v, q_len, k_len, scale, dtype, out, lse, w=None, w0=None, decay=0.0, prompt=False):
    """Against the formula.  Let A be a row's sum of |q k| scale over the dims (its largest over the keys).  Scores: the
    products are exact (fp32 queries to 2^-22 of each), sums of up to 128 of them in the tensor core, cut off at a few
    2^-24 of their size for each of at most 16 steps, and two roundings of the scale: 2^-19 A at most.  A weight is then off by
    d = 2^-19 A + 2^-20 of itself (exp2 and its argument), the sum of them by as much, and goes into the product rounded (r:
    half an fp16 step 2^-11, of two halves 2^-21; prompts of bf16 2^-8) or to fp16's smallest step, 2^-24 of weights times 2^6 to 2^14: half of it is 2^-31
    of the row's largest weight, which is 1 at most, so that an output is off by 2^-31 sum |v| more.  The product's running sum loses 2^-23 of its size per step, 2^-17 over the 64 steps that a warp takes here.  Prompts of fp32
    go through chains of 64 fused multiply-adds for a score (2^-17 A with the rest) and of up to 400 for an output (2^-15)."""
    at, rows = 0, 0
    f32 = dtype == F32
    r = 2.0 ** -21 if f32 else 2.0 ** -8 if prompt else 2.0 ** -11
    for i, (n, kl) in enumerate(zip(q_len, k_len)):
        o, z, wt, A, mag, flat = F.attend(q[rows:rows + n], k[at:at + kl], v[at:at + kl], n, kl, scale)
        d = 2.0 ** (-17 if prompt else -19) * A + 2.0 ** -20
        got, gz = out[rows:rows + n].double().cpu(), lse[rows:rows + n].double().cpu()
        tol = torch.finfo(dtype).eps / 2 * o.abs() + (2 * d[..., None] + r + 2.0 ** (-15 if prompt else -17)) * mag + 2.0 ** -31 * flat + 1e-30
        assert bool(((got - o).abs() <= tol).all()), (i, float(((got - o).abs() / tol).max()))
        fin = z > -math.inf
        assert torch.equal(gz == -math.inf, ~fin)
        assert bool(((gz - z).abs()[fin] <= (d + 2.0 ** -22 * (1 + z.abs()))[fin]).all())
        if w is not None and n:
            # each row's weight is off by the score's and the sum's error and 2^-20 of itself; decay adds a rounding
            want = wt + (decay * w0[i, :, :kl].double().cpu() if decay else 0)
            e = (2 * float(d.max()) + 2.0 ** -19 * (1 + float(z.abs().max()))) * wt + 2.0 ** -23 * want.abs()
            assert bool(((w[i, :, :kl].double().cpu() - want).abs() <= e + 1e-37).all())
        if w is not None:
            k_from = kl if n else 0
            assert torch.equal(w[i, :, k_from:], w0[i, :, k_from:])
        at += kl
        rows += n


def run(q_len, k_len, hq, hk, d, page, dtype, weigh=False, decay=0.5, scale=None, seed=1, ks=1.0, vs=1.0, strided=False,
        k_size=1.0):
    g = gen(seed)
    cache, table = make(k_len, page, hk, d, seed, ks, vs)
    k, v = fill(cache, table, k_len, dtype, g, k_size)
    rows = sum(q_len) + 2
    if strided:
        buf = randn((rows, hq + 3, d + 16), dtype, g)
        q = buf[:, 1:1 + hq, :d]
    else:
        q = randn((rows, hq, d), dtype, g)
    lse = torch.full((rows, hq), 7.0, device="cuda")
    out = torch.full((rows, hq, d), 7.0, dtype=dtype, device="cuda")
    w = w0 = None
    if weigh:
        w = torch.rand((len(k_len), hk, max(k_len) + 5), device="cuda", generator=g)
        w0 = w.clone()
        if decay == 0:
            w[:] = math.nan
            for i, n in enumerate(k_len):
                w[i, :, n if q_len[i] else 0:] = w0[i, :, n if q_len[i] else 0:]
    got = cache.attend(q, table, q_len, k_len, scale=scale, out=out, lse=lse, weights=w, decay=decay)
    assert got is out
    prompt = max(q_len) * (hq // hk) > 64
    check(q, k, v, q_len, k_len, d ** -0.5 if scale is None else scale, dtype, out, lse, w, w0, decay, prompt)
    assert bool((out[-2:] == 7).all()) and bool((lse[-2:] == 7).all())
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("q_len,k_len,hq,hk,d,page", [
    ([1], [1], 1, 1, 64, 16), ([1], [16], 4, 1, 128, 16), ([1], [17], 8, 1, 64, 64), ([1, 1, 1], [33, 0, 700], 4, 4, 128, 32),
    ([1, 0, 1], [64, 50, 65], 6, 2, 128, 64), ([1], [5003], 16, 1, 128, 256), ([1, 1], [3000, 2], 9, 3, 64, 128),
    ([2, 1, 5], [2, 900, 1300], 4, 2, 128, 64), ([4], [4], 16, 1, 64, 16), ([7, 3], [130, 3], 8, 8, 64, 1024),
    ([3, 6], [1, 4], 2, 1, 128, 16), ([8], [333], 8, 1, 128, 64), ([16, 1], [100, 70], 4, 1, 64, 32)])
def test_attend(q_len, k_len, hq, hk, d, page, weigh, dtype):
    run(q_len, k_len, hq, hk, d, page, dtype, weigh)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(scale=-0.3), dict(scale=0.0), dict(scale=3.0, k_size=2.0), dict(ks=2.0, vs=0.125), dict(decay=0.0),
                                dict(decay=1.0), dict(strided=True), dict(decay=-0.25, ks=0.25)])
def test_attend_scales_strides_and_decay(kw, dtype):
    run([1, 2, 1], [40, 555, 2100], 8, 2, 64, 32, dtype, True, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_len,k_len,hq,hk,d", [([70], [70], 1, 1, 64), ([40, 1, 90], [200, 300, 111], 4, 2, 128),
                                                 ([1, 80, 0, 65, 1], [9, 80, 7, 400, 100], 2, 1, 64),
                                                 ([80, 100], [20, 0], 1, 1, 128)])
def test_attend_prompts(q_len, k_len, hq, hk, d, dtype):
    """Segments that are read back, beside single tokens."""
    run(q_len, k_len, hq, hk, d, 32, dtype)


def test_large_and_small_queries():
    """Rows whose values are far from 1: products stay within the range of their type."""
    g = gen(9)
    cache, table = make([300], 64, 2, 128)
    k, v = fill(cache, table, [300], BF, g)
    for dtype in (BF, F32):
        q = randn((6, 4, 128), dtype, g)
        sizes = torch.tensor([1e30, 1e-30, 0.0, 3e4, 1e-38, 1.0], device="cuda")
        q = (q.float() * sizes[:, None, None]).to(dtype)
        for j, s in enumerate(sizes.tolist()):
            scale = 0.05 / s if 1e-37 < s else 1.0
            lse = torch.empty((1, 4), device="cuda")
            out = cache.attend(q[j:j + 1], table, [1], [300], scale=scale, lse=lse)
            check(q[j:j + 1], k, v, [1], [300], scale, dtype, out, lse)
    ok()


def test_nan_where_it_is_seen():
    g, T = gen(11), 100
    cache, table = make([T, T], 32, 1, 64)
    k, v = (randn((2 * T, 1, 64), BF, g) for _ in range(2))
    k[40, 0, 3], v[T + 60, 0, 20] = math.nan, math.inf
    cache.store(k, v, table, [0, 0], [T, T])
    q = randn((8, 4, 64), BF, g)
    w = torch.zeros((2, 1, T), device="cuda")
    lse = torch.empty((8, 4), device="cuda")
    out = cache.attend(q, table, [4, 4], [T, T], lse=lse, weights=w, decay=0.0)
    assert bool(out[:4].isnan().all()) and bool(lse[:4].isnan().all()) and bool(w[0].isnan().all())
    assert bool(out[4:, :, 16:32].isnan().all()) and not bool(out[4:, :, :16].isnan().any())
    assert not bool(lse[4:].isnan().any()) and not bool(w[1].isnan().any())
    # places behind a segment's tokens may hold anything
    out = cache.attend(q[:2], table, [1, 1], [40, 60], lse=lse[:2])
    assert not bool(out.isnan().any()) and not bool(lse[:2].isnan().any())
    # a query that is NaN or infinite makes its own row NaN and no other
    q[1, 2, 5], q[2, 0, 7] = math.nan, math.inf
    out = cache.attend(q[:4], table[1:], [4], [59])
    bad = out.isnan().all(-1)
    assert bad.nonzero().tolist() == [[1, 2], [2, 0]] and int(out.isnan().any(-1).sum()) == 2
    ok()


# ---- eviction -----------------------------------------------------------------


def kept(w, n, keep, sink, recent):
    """The places that stay, from the weights of one segment and head."""
    if n <= keep:
        return np.arange(n)
    r = w[:n].astype(np.float64)
    r = np.where(np.isnan(r), np.inf, r)
    nan = np.isnan(w[:n])
    must = np.zeros(n, bool)
    must[:sink] = True
    must[n - recent:] = True
    order = np.lexsort((np.arange(n), -r, ~nan, ~must))
    return np.sort(order[:keep])


@pytest.mark.parametrize("d,hk,page", [(64, 1, 16), (128, 3, 64), (64, 2, 256), (128, 1, 32)])
@pytest.mark.parametrize("lens,keep,sink,recent", [([50], 49, 0, 0), ([50, 7, 300], 33, 4, 8), ([200, 0, 64], 64, 0, 64), ([90], 1, 0, 0),
                                                   ([700, 701, 5000], 401, 1, 200), ([20000], 3001, 4, 100), ([33, 40], 40, 40, 0)])
def test_evict(lens, keep, sink, recent, d, hk, page):
    g = gen(keep + d)
    spare = sum(-(-min(n, keep) // page) + 1 for n in lens)
    cache, table = make(lens, page, hk, d, spare=spare)
    k, v = fill(cache, table, lens, BF, g)
    used = set(int(x) for i, n in enumerate(lens) for x in table[i, :max(1, -(-n // page))].tolist())
    free = [i for i in range(cache.pages.shape[0]) if i not in used]
    width = max(1, -(-min(max(lens), keep) // page))
    out_table = torch.tensor(free[:len(lens) * width] if len(free) >= len(lens) * width else (free * 99)[:len(lens) * width],
                             dtype=torch.int32)
    at = 0
    out_table = torch.zeros((len(lens), width), dtype=torch.int32)
    for i, n in enumerate(lens):
        m = -(-min(n, keep) // page)
        out_table[i, :m] = torch.tensor(free[at:at + m], dtype=torch.int32)
        at += m
    out_table = out_table.cuda()
    w = torch.exp(3 * torch.randn((len(lens), hk, max(lens) + 3), device="cuda", generator=g)).bfloat16().float()
    w[..., ::5] = 0.0
    w[..., 1::15] = -0.0
    if hk > 1:
        w[:, 1] = 1.0  # all alike: the lowest places stay
        w[:, 1, 10::20] = math.nan
    before = cache.pages.clone()
    ow = torch.full((len(lens), hk, keep + 9), 5.0, device="cuda")
    index, got = cache.evict(table, lens, w, keep, out_table, sink, recent, out_weights=ow)
    assert got is ow
    wn, at = w.cpu().numpy(), 0
    for i, n in enumerate(lens):
        m = min(n, keep)
        k2, v2 = cache.load(out_table[i:i + 1], [0], [m], dtype=F32)
        for h in range(hk):
            idx = kept(wn[i, h], n, keep, sink, recent)
            assert index[i, h].tolist() == idx.tolist() + [-1] * (keep - m), (i, h)
            assert same(ow[i, h, :m], w[i, h, idx]) and bool((ow[i, h, m:] == 0).all())
            assert same(k2[:, h], k[at + idx, h]) and same(v2[:, h], v[at + idx, h])
        at += n
    for p in used:  # the pages that were read stay as they were
        assert torch.equal(before[p], cache.pages[p])
    plain = cache.evict(table, lens, w, keep, out_table, sink, recent)
    assert torch.equal(plain[0], index) and same(plain[1], ow[..., :keep])
    ok()


# ---- as they are used ------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_layer_as_a_model_runs_it(dtype):
    """A prompt's rows normed, rotated by three axes, stored and attended to; its last queries' weights choose what stays;
    then steps that norm, rotate, store and attend behind it, each against the formula over what the cache holds."""
    g, hq, hk, d, page, T, keep = gen(21), 8, 2, 64, 32, 300, 120
    table_of = K.rope_table(d)
    axes = [0] * 8 + [1] * 12 + [2] * 12
    cache, table = make([T, T - 77], page, hk, d, spare=12)
    lens = [T, T - 77]
    used = set(table.flatten().tolist())
    free = [i for i in range(cache.pages.shape[0]) if i not in used]
    out_table = torch.tensor(free[:10], dtype=torch.int32, device="cuda").view(2, 5)

    def rows(n):
        x = randn((n, hq + 2 * hk, d), dtype, g)
        pos = torch.randint(0, 500, (n, 3), device="cuda", generator=g)
        K.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], pos, table_of, axes=axes, out_q=x[:, :hq], out_k=x[:, hq:hq + hk])
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]

    def held(t, n):
        k, v = cache.load(t, [0] * len(n), n, dtype=F32)
        return k.double().cpu(), v.double().cpu()

    q, k, v = rows(sum(lens))
    cache.store(k, v, table, [0, 0], lens)
    k2, v2 = held(table, lens)
    assert same(k2, F.held(k)) and same(v2, F.held(v))
    lse = torch.empty((sum(lens), hq), device="cuda")
    out = cache.attend(q, table, lens, lens, lse=lse)
    check(q, k2, v2, lens, lens, d ** -0.5, dtype, out, lse, prompt=True)
    w = torch.zeros((2, hk, keep + 10), device="cuda")
    seen = torch.zeros((2, hk, T), device="cuda")
    last = [slice(lens[0] - 16, lens[0]), slice(sum(lens) - 16, sum(lens))]
    cache.attend(torch.cat([q[s] for s in last]), table, [16, 16], lens, weights=seen, decay=0.0)
    index, _ = cache.evict(table, lens, seen, keep, out_table, n_sink=4, n_recent=16, out_weights=w)
    k3, v3 = held(out_table, [keep, keep])
    for b in range(2):
        for h in range(hk):
            idx = index[b, h].cpu() + (0 if b == 0 else T)
            assert same(k3[b * keep:(b + 1) * keep, h], k2[idx.long(), h]) and same(v3[b * keep:(b + 1) * keep, h], v2[idx.long(), h])
    for t in range(keep, keep + 10):
        q, k, v = rows(2)
        cache.store(k, v, out_table, [t, t], [1, 1])
        w0, lse = w.clone(), torch.empty((2, hq), device="cuda")
        out = cache.attend(q, out_table, [1, 1], [t + 1, t + 1], lse=lse, weights=w, decay=0.875)
        kk, vv = held(out_table, [t + 1, t + 1])
        check(q, kk, vv, [1, 1], [t + 1, t + 1], d ** -0.5, dtype, out, lse, w, w0, 0.875)
    ok()


def test_a_captured_call_replays():
    """Store, attention with weights and eviction in one graph; two graphs of their own workspaces on two streams."""
    g, hk, d, page, T = gen(31), 2, 128, 64, 900
    cache, table = make([T, T], page, hk, d, spare=20)
    k, v = fill(cache, table, [T, T], BF, g)
    free = [i for i in range(cache.pages.shape[0]) if i not in set(table.flatten().tolist())]
    outs = [torch.tensor(free[10 * i:10 * i + 10], dtype=torch.int32, device="cuda").view(2, 5) for i in range(2)]
    q = randn((6, 8, d), BF, g)
    nk, nv = randn((2, hk, d), BF, g), randn((2, hk, d), BF, g)
    state = [dict(out=torch.zeros_like(q), w=torch.zeros((2, hk, T), device="cuda"), ow=torch.zeros((2, hk, 300), device="cuda"),
                  index=torch.zeros((2, hk, 300), dtype=torch.int32, device="cuda"),
                  space=torch.empty(cache.workspace(q, table, [3, 3], [T, T], weights=torch.zeros((2, hk, T), device="cuda")),
                                    dtype=torch.uint8, device="cuda")) for _ in range(3)]

    def call(s, t):
        cache.attend(q, table, [3, 3], [T, T], out=s["out"], weights=s["w"], decay=0.0, workspace=s["space"])
        cache.evict(table, [T, T], s["w"], 300, t, 2, 20, index=s["index"], out_weights=s["ow"])

    cache.store(nk, nv, table, [T - 1, T - 1], [1, 1])
    call(state[2], outs[0])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            cache.store(nk, nv, table, [T - 1, T - 1], [1, 1])
            call(state[i], outs[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for x in ("out", "w", "ow", "index"):
            assert torch.equal(state[i][x], state[2][x]), x
    ok()


def test_other_streams_and_the_same_bits_every_time():
    g, hk, d, page = gen(41), 4, 64, 32
    lens = [1, 700, 5000, 64]
    cache, table = make(lens, page, hk, d)
    fill(cache, table, lens, BF, g)
    q = randn((4, 16, d), BF, g)
    w = torch.zeros((4, hk, 5000), device="cuda")
    want = cache.attend(q, table, [1] * 4, lens, weights=w, decay=0.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for i in range(20):
        w2 = torch.zeros_like(w)
        torch.cuda.synchronize()
        if i % 2:
            got = cache.attend(q, table, [1] * 4, lens, weights=w2, decay=0.0, stream=s)
            k = cache.load(table, [0] * 4, lens, stream=s)[0]
        else:
            with torch.cuda.stream(s):
                got = cache.attend(q, table, [1] * 4, lens, weights=w2, decay=0.0)
                k = cache.load(table, [0] * 4, lens)[0]
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(w, w2) and k.shape[0] == sum(lens)
    ok()


@pytest.mark.parametrize("weigh", [False, True])
def test_many_segments(weigh):
    """More segments than a launch takes, prompts among them."""
    g, hk, d, page, n = gen(51), 1, 64, 16, 600
    r = np.random.RandomState(2)
    lens = r.randint(0, 90, n).tolist()
    q_len = r.choice([0, 1, 1, 1, 2], n).tolist()
    if not weigh:
        q_len[5] = q_len[6] = q_len[300] = 80
    cache, table = make(lens, page, hk, d)
    k, v = fill(cache, table, lens, BF, g)
    q, lse = randn((sum(q_len), 1, d), BF, g), torch.empty((sum(q_len), 1), device="cuda")
    w = torch.rand((n, hk, 90), device="cuda", generator=g) if weigh else None
    w0 = w.clone() if weigh else None
    out = cache.attend(q, table, q_len, lens, lse=lse, weights=w, decay=0.5)
    check(q, k, v, q_len, lens, 0.125, BF, out, lse, w, w0, 0.5, prompt=not weigh)
    ok()


def test_bad_page_ids_are_flagged():
    g, hk, d = gen(61), 2, 64
    cache, table = make([64, 64], 16, hk, d)
    k, v = fill(cache, table, [64, 64], BF, g)
    before = cache.pages.clone()
    bad = table.clone()
    bad[0, 1], bad[1, 3] = cache.pages.shape[0], -7
    cache.store(randn((64, hk, d), BF, g), randn((64, hk, d), BF, g), bad[:1], [0], [64])
    assert K.window_check() == (K.ERR_DEVICE_CHECK, 2)
    cache.pages.copy_(before)
    k2, v2 = cache.load(bad, [0, 0], [64, 64], dtype=F32)
    assert K.window_check() == (K.ERR_DEVICE_CHECK, 2)
    k[16:32] = v[16:32] = k[112:] = v[112:] = 0
    assert same(k2, k) and same(v2, v)
    cache.attend(randn((2, 4, d), BF, g), bad, [1, 1], [64, 64])
    assert K.window_check() == (K.ERR_DEVICE_CHECK, 2)
    cache.attend(randn((2, 4, d), BF, g), bad, [1, 1], [16, 48])  # (entries behind the tokens are not looked at)
    ok()
    outs = torch.full((2, 4), 1 << 30, dtype=torch.int32, device="cuda")
    cache.evict(table, [64, 64], torch.zeros((2, hk, 64), device="cuda"), 40, outs)
    assert K.window_check() == (K.ERR_DEVICE_CHECK, 2)
    assert torch.equal(cache.pages, before)


def test_refusals():
    g, hk, d = gen(71), 2, 64
    cache, table = make([64, 64], 16, hk, d)
    k = randn((64, hk, d), BF, g)
    with pytest.raises(ValueError):
        K.Kv4Cache(cache.pages[:, :-16], hk, d, 16)
    with pytest.raises(ValueError):
        K.Kv4Cache(cache.pages.cpu(), hk, d, 16)
    for args in ((k.half(), k.half(), table), (k, k[:5], table), (k, k, table.long()), (k, k, table.cpu()), (k, k, table[0]),
                 (k[:, :, :32], k[:, :, :32], table), (k.cpu(), k.cpu(), table), (k, k, table[:0])):
        with pytest.raises(ValueError):
            cache.store(*args, [0], [64])
    with pytest.raises(ValueError):
        cache.store(k, k, table, [0, 0], [64])
    with pytest.raises(ValueError):
        cache.store(k, k, table, [0.5], [64])
    for start, n in (([60], [5]), ([-1], [2]), ([0], [65])):
        with pytest.raises(K.KvpoolError):
            cache.store(k, k, table, start, n)
    with pytest.raises(K.KvpoolError):
        cache.store(k[:, :1], k[:, :1], table, [0], [1])
    q = randn((4, 4, d), BF, g)
    for kw in (dict(lse=torch.zeros(4, 2, device="cuda")), dict(weights=torch.zeros(2, hk, 63, device="cuda")),
               dict(weights=torch.zeros(2, 1, 64, device="cuda")), dict(out=q.float()), dict(out=q[:3])):
        with pytest.raises(ValueError):
            cache.attend(q, table, [2, 2], [64, 64], **kw)
    for kw in (dict(out=q.flip(0)[:4].as_strided((4, 4, d), (0, d, 1))),):
        with pytest.raises(ValueError):
            cache.attend(q, table, [2, 2], [64, 64], **kw)
    with pytest.raises((ValueError, K.KvpoolError)):  # (no fp32 number)
        cache.attend(q, table, [2, 2], [64, 64], scale=1e300)
    with pytest.raises(K.KvpoolError):
        cache.attend(q, table, [2, 2], [64, 64], workspace=torch.empty(0, dtype=torch.uint8, device="cuda"),
                     weights=torch.zeros(2, hk, 64, device="cuda"))
    w = torch.zeros(2, hk, 64, device="cuda")
    with pytest.raises(K.KvpoolError):
        cache.evict(table, [64, 64], w, 40, table, out_weights=w)
    with pytest.raises(ValueError):
        cache.evict(table, [64, 64], w, 40, table, index=torch.zeros(2, hk, 39, dtype=torch.int32, device="cuda"))
    ok()


@pytest.mark.parametrize("q_len,k_len,hq,hk", [([1, 3], [500, 40], 8, 2), ([1], [9000], 4, 1), ([1] * 40, [3000] * 40, 16, 4),
                                               ([70, 1], [200, 100], 2, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_outputs_over_the_queries(q_len, k_len, hq, hk, dtype):
    g = gen(81)
    cache, table = make(k_len, 64, hk, 64)
    fill(cache, table, k_len, dtype, g)
    rows = randn((sum(q_len), hq + 2, 64), dtype, g)
    q = rows[:, 1:-1]
    want = cache.attend(q, table, q_len, k_len)
    assert cache.attend(q, table, q_len, k_len, out=q) is q and torch.equal(q, want)
    ok()


def test_weights_in_either_order():
    """Accumulators [key heads][segments][places] seen as [segments][key heads][places]."""
    g, lens = gen(83), [100, 333, 2]
    cache, table = make(lens, 16, 4, 64)
    fill(cache, table, lens, BF, g)
    q = randn((3, 8, 64), BF, g)
    a, b = torch.zeros((3, 4, 333), device="cuda"), torch.zeros((4, 3, 340), device="cuda")
    cache.attend(q, table, [1] * 3, lens, weights=a)
    cache.attend(q, table, [1] * 3, lens, weights=b.transpose(0, 1))
    assert torch.equal(a, b.transpose(0, 1)[..., :333]) and bool((b[..., 333:] == 0).all())
    with pytest.raises(K.KvpoolError):
        cache.attend(q, table, [1] * 3, lens, weights=b[:, :1].expand(4, 3, 340).transpose(0, 1))
    ok()


def test_shared_pages_are_read():
    """Two requests behind one prefix: their tables name the same pages; eviction leaves them to both."""
    g, hk, d, page = gen(85), 2, 128, 16
    cache, table = make([160, 32, 0, 0], page, hk, d, spare=12)
    used = set(table.flatten().tolist())
    free = [i for i in range(cache.pages.shape[0]) if i not in used]
    rows = torch.zeros((2, 12), dtype=torch.int32, device="cuda")
    rows[0, :10] = rows[1, :10] = table[0, :10]
    rows[1, 10:] = table[1, :2]
    k, v = randn((192, hk, d), BF, g), randn((192, hk, d), BF, g)
    cache.store(k[:160], v[:160], rows[:1], [0], [160])
    cache.store(k[160:], v[160:], rows[1:], [160], [32])
    hk_, hv_ = F.held(k), F.held(v)
    q, lse, w = randn((2, 4, d), BF, g), torch.empty((2, 4), device="cuda"), torch.zeros((2, hk, 192), device="cuda")
    out = cache.attend(q, rows, [1, 1], [160, 192], lse=lse, weights=w, decay=0.0)
    both = [torch.cat([x[:160], x]) for x in (hk_, hv_)]
    check(q, *both, [1, 1], [160, 192], d ** -0.5, BF, out, lse, w, torch.zeros_like(w))
    before = cache.pages.clone()
    outs = torch.tensor(free[:8], dtype=torch.int32, device="cuda").view(2, 4)
    cache.evict(rows, [160, 192], w, 64, outs)
    for p in used:
        assert torch.equal(cache.pages[p], before[p])
    assert torch.equal(cache.attend(q, rows, [1, 1], [160, 192]), out)
    ok()


def test_pages_past_32_bits():
    g, hk, d, page = gen(87), 2, 64, 1024
    size = K.kv4_page_bytes(hk, d, page)
    n = (1 << 32) // size + 4
    pages = torch.empty((n, size), dtype=torch.uint8, device="cuda")
    cache = K.Kv4Cache(pages, hk, d, page)
    table = torch.tensor([[n - 1, 0, n - 2]], dtype=torch.int32, device="cuda")
    outs = torch.tensor([[n - 3]], dtype=torch.int32, device="cuda")
    k, v = fill(cache, table, [3000], BF, g)
    q, lse, w = randn((1, 4, d), BF, g), torch.empty((1, 4), device="cuda"), torch.zeros((1, hk, 3000), device="cuda")
    out = cache.attend(q, table, [1], [3000], lse=lse, weights=w)
    check(q, k, v, [1], [3000], 0.125, BF, out, lse, w, torch.zeros_like(w))
    index, _ = cache.evict(table, [3000], w, 1000, outs)
    k2, v2 = cache.load(outs, [0], [1000], dtype=F32)
    for h in range(hk):
        assert same(k2[:, h], k[index[0, h].cpu().long(), h]) and same(v2[:, h], v[index[0, h].cpu().long(), h])
    ok()


def test_evict_from_more_tokens_than_shared_memory_holds():
    g, n, keep = gen(89), 450_000, 700
    cache, table = make([n], 1024, 1, 64, spare=1)
    used = set(table.flatten().tolist())
    outs = torch.tensor([[i for i in range(cache.pages.shape[0]) if i not in used]], dtype=torch.int32, device="cuda")
    k, _ = fill(cache, table, [n], BF, g)
    w = torch.rand((1, 1, n), device="cuda", generator=g).bfloat16().float()
    index, left = cache.evict(table, [n], w, keep, outs, 4, 50)
    idx = kept(w[0, 0].cpu().numpy(), n, keep, 4, 50)
    assert index[0, 0].tolist() == idx.tolist() and torch.equal(left[0, 0], w[0, 0, idx])
    assert same(cache.load(outs, [0], [keep], dtype=F32)[0][:, 0], k[idx, 0])
    ok()


def test_evict_many_segments():
    g, n, keep = gen(91), 300, 20
    lens = np.random.RandomState(1).randint(0, 60, n).tolist()
    cache, table = make(lens, 16, 1, 64, spare=2 * n)
    used = set(int(x) for i, m in enumerate(lens) for x in table[i, :max(1, -(-m // 16))].tolist())
    free = [i for i in range(cache.pages.shape[0]) if i not in used]
    outs = torch.tensor(free[:2 * n], dtype=torch.int32, device="cuda").view(n, 2)
    k, _ = fill(cache, table, lens, BF, g)
    w = torch.rand((n, 1, 60), device="cuda", generator=g)
    index, left = cache.evict(table, lens, w, keep, outs, 2, 5)
    got = cache.load(outs, [0] * n, [min(m, keep) for m in lens], dtype=F32)[0]
    at = to = 0
    for i, m in enumerate(lens):
        idx = kept(w[i, 0].cpu().numpy(), m, keep, 2, 5)
        assert index[i, 0].tolist() == idx.tolist() + [-1] * (keep - len(idx))
        assert same(got[to:to + len(idx), 0], k[at + idx, 0])
        at, to = at + m, to + len(idx)
    ok()


FIRST = """
import sys; sys.path.insert(0, {root!r})
import torch
from heterogeneous_compressed_kv_gb300 import kvpool as K
n = 2000
cache = K.Kv4Cache(torch.zeros((40, K.kv4_page_bytes(2, 64, 64)), dtype=torch.uint8, device="cuda"), 2, 64, 64)
table = torch.arange(32, dtype=torch.int32, device="cuda")[None]
outs = torch.arange(32, 40, dtype=torch.int32, device="cuda")[None]
k = torch.randn((n, 2, 64), device="cuda").bfloat16()
q = torch.randn(({rows}, 8, 64), device="cuda").bfloat16()
w = torch.zeros((1, 2, n), device="cuda") if {rows} < 16 else None
index = torch.zeros((1, 2, 500), dtype=torch.int32, device="cuda")
left = torch.zeros((1, 2, 500), device="cuda")
out = torch.zeros_like(q)
def call():
    cache.store(k, k, table, [0], [n])
    cache.attend(q, table, [{rows}], [n], out=out, weights=w, decay=0.0)
    if w is not None:
        cache.evict(table, [n], w, 500, outs, index=index, out_weights=left)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
first = [x.clone() for x in (out, index, left)]
assert float(first[0].float().abs().sum()) > 0
call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (out, index, left)))
assert K.window_check() == (K.OK, 0)
"""


@pytest.mark.parametrize("rows", [1, 40])
def test_the_first_calls_of_a_process_inside_a_capture(rows):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, rows=rows)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_at_once():
    import threading
    g, hk, d, lens = gen(93), 2, 64, [3000, 50, 700]
    cache, table = make(lens, 64, hk, d)
    fill(cache, table, lens, BF, g)
    q = randn((5, 8, d), BF, g)
    args = (q, table, [1, 3, 1], lens)
    w0 = torch.zeros((3, hk, 3000), device="cuda")
    want, back = cache.attend(*args, weights=w0, decay=0.0), cache.load(table, [0] * 3, lens)[0]
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = []
            for _ in range(20):
                w = torch.zeros_like(w0)
                got.append((cache.attend(*args, weights=w, decay=0.0), w, cache.load(table, [0] * 3, lens)[0]))
            s.synchronize()
            bad.extend(1 for a, b, c in got if not (torch.equal(a, want) and torch.equal(b, w0) and torch.equal(c, back)))
            s.synchronize()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    ok()


@pytest.mark.parametrize("q_len,lens,hq,hk,dtype", [([1], [20000], 16, 1, BF), ([1] * 8, [7000] * 8, 16, 4, BF), ([2], [9000], 8, 1, BF),
                                                    ([1] * 60, [130] * 60, 8, 2, BF), ([5], [6000], 4, 2, F32), ([1] * 3, [9000, 20, 400], 8, 8, F32)])
def test_both_forms_in_many_parts(q_len, lens, hq, hk, dtype):
    """Long units in hundreds of shares, short ones in a CTA each."""
    run(q_len, lens, hq, hk, 128, 64, dtype, True)
    run(q_len, lens, hq, hk, 128, 16, dtype, False)


def test_every_largest_value_and_its_borders():
    """Groups of every positive bf16 largest value, their other values the borders between codes and their neighbours."""
    bits = np.arange(1, 0x7F80, dtype=np.uint16)
    bits = bits[:len(bits) // 8 * 8]
    amax = torch.from_numpy(bits.view(np.int16)).view(BF)
    s = F.nearest((amax.float().numpy() / np.float32(6)).astype(np.float64), F.E4M3)
    border = torch.from_numpy(s)[:, None] * torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    near = border.to(BF)
    assert bool((near.double() == border)[s > 2.0 ** -9].all())
    pad = near[:, :1] * 0
    up, down = (torch.where(near > 0, (near.view(torch.int16) + d).view(BF), near) for d in (1, -1))
    for other, dtype in ((up, BF), (down, BF), (up, F32), (down, F32)):
        x = torch.cat([amax[:, None], near, -other, pad], 1).reshape(-1, 1, 128).to(dtype).cuda()
        n = x.shape[0]
        cache, table = make([n], 64, 1, 128)
        cache.store(x, x.flip(0), table, [0], [n])
        k, v = cache.load(table, [0], [n], dtype=F32)
        assert same(k, F.held(x)) and same(v, F.held(x.flip(0)))
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_len,k_len,hq,hk,d", [([200], [200], 4, 1, 64), ([33, 1, 150], [40, 900, 333], 4, 2, 128), ([300], [1500], 2, 2, 64)])
def test_prompts_that_are_not_read_back(q_len, k_len, hq, hk, d, dtype):
    """Short enough for the kernel of single tokens (fp32 ones always go there)."""
    run(q_len, k_len, hq, hk, d, 16, dtype)
    run(q_len, k_len, hq, hk, d, 128, dtype, strided=True)


def test_long_prompts_of_bf16_are_read_back():
    g, d, hk = gen(97), 64, 1
    cache, table = make([9000], 64, hk, d)
    k, v = fill(cache, table, [9000], BF, g)
    q, lse = randn((600, 8, d), BF, g), torch.empty((600, 8), device="cuda")
    assert cache.workspace(q, table, [600], [9000]) >= 2 * 9000 * hk * d * 2
    out = cache.attend(q, table, [600], [9000], lse=lse)
    # the last 40 queries alone, by the other kernel
    want_lse = torch.empty((40, 8), device="cuda")
    want = cache.attend(q[-40:], table, [40], [9000], lse=want_lse)
    # weights rounded to bf16 (2^-8 of each) against fp16's, both outputs rounded
    assert float((out[-40:].double() - want.double()).norm() / want.double().norm()) < 2.0 ** -7
    assert float((lse[-40:] - want_lse).abs().max()) < 1e-4
    ok()
