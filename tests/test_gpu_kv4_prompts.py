"""Long bf16 segments over the 4-bit paged cache: those whose tokens are read back to rows before they are attended to.
Against the formulas in 64 bits, over what the cache holds."""
import math

import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests.test_gpu_kv4 import BF, F32, fill, gen, make, ok, randn

pytestmark = pytest.mark.gpu


def held(cache, table, lens):
    """What the cache holds of every segment's tokens, in float64."""
    k, v = cache.load(table, [0] * len(lens), lens, dtype=F32)
    return k.double(), v.double()


def rows64(q, pos, k, v, scale):
    """(out, lse, A, mag, flat) of query rows q [n][hq][d] at places pos over k and v [keys][hk][d], in float64: A the
    largest sum |q k| |scale| of a row, mag the sum p |v|, flat the sum |v| over what the row sees."""
    n, hq, d = q.shape
    G = hq // k.shape[1]
    t = torch.arange(k.shape[0], device=q.device)
    hidden = t[None] > pos[:, None]
    none = pos < 0 if k.shape[0] else torch.ones_like(pos, dtype=torch.bool)
    res = [[] for _ in range(5)]
    for h in range(hq):
        kh, vh, qh = k[:, h // G], v[:, h // G], q[:, h].double()
        s = (qh @ kh.T * scale).masked_fill(hidden, -math.inf)
        z = torch.logsumexp(s, -1) if k.shape[0] else torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
        p = torch.where(hidden | none[:, None], 0.0, torch.exp(s - torch.where(none, 0.0, z)[:, None]))
        size = (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(hidden, 0.0)
        for x, y in zip(res, (p @ vh, z, size.amax(-1) if k.shape[0] else torch.zeros_like(z), p @ vh.abs(),
                              (~hidden).double() @ vh.abs())):
            x.append(y)
    return [torch.stack(x, 1) for x in res]


def bounds(o, z, A, mag, flat, keys, r):
    """(output tolerance, log-sum-exp tolerance).  A score's products are exact; their sum, taken in the tensor core in steps
    of 16, is off by less than 2^-19 A, with the scale's roundings less than 2^-17 A; a weight by as much and 2^-20 of itself
    (exp2 and its argument), and by r where it is rounded for its product (half an fp16 or bf16 step: 2^-11 or 2^-8) or by
    half of fp16's smallest step against weights of 2^6 and more (2^-31 of the row's largest, at most 1, for every value).
    The running sum of outputs cuts off 2^-23 of itself at each step of 16 keys; the weights' sum takes 32 of a tile by
    one after the other, the tiles after each other and the parts (fewer than 64)."""
    d = 2.0 ** -17 * A + 2.0 ** -20
    sums = 2.0 ** -24 * (keys / 128 + 128)
    tol = 2.0 ** -8 * o.abs() + (2 * d[..., None] + r + 2.0 ** -23 * (keys / 16 + 64) + sums) * mag + 2.0 ** -31 * flat + 1e-30
    return tol, d + sums + 2.0 ** -22 * (1 + z.abs())


def check(q, k, v, q_len, k_len, scale, out, lse, r=2.0 ** -8, most=400):
    """Every row of segments of up to `most` queries; of longer ones the first and the last, and every 50th between (of
    more than 5,000 queries, every 2,050th)."""
    at = row = 0
    for i, (n, kl) in enumerate(zip(q_len, k_len)):
        for j0 in range(0, n, 100):
            j = torch.arange(j0, min(n, j0 + 100), device="cuda")
            if n > most and 0 < j0 and j0 + 100 < n:
                if n > 5000 and j0 // 100 % 41:
                    continue
                j = j[::50]
            o, z, A, mag, flat = rows64(q[row + j], kl - n + j, k[at:at + kl], v[at:at + kl], scale)
            tol, ztol = bounds(o, z, A, mag, flat, kl, r)
            got, gz = out[row + j].double(), lse[row + j].double()
            assert bool(((got - o).abs() <= tol).all()), (i, j0, float(((got - o).abs() / tol).max()))
            fin = z > -math.inf
            assert torch.equal(gz == -math.inf, ~fin)
            assert bool(((gz - z).abs() <= ztol)[fin].all()), (i, j0)
            assert bool((got[~fin] == 0).all())
        at += kl
        row += n


def rows_read_back(cache, q, table, q_len, k_len, at_least, **kw):
    """Does the call's workspace have room for the keys and values of so many tokens as bf16 rows?"""
    return cache.workspace(q, table, q_len, k_len, **kw) >= at_least * cache.kv_heads * cache.head_dim * 4


SHAPES = [  # q_len, k_len, query heads, key heads, dim, page, tokens of the longest run of prompts
    ([1, 300, 0, 200, 1, 150], [50, 4000, 30, 2500, 700, 150], 8, 2, 128, 16, 6500),
    ([100, 5], [8000, 8000], 16, 1, 64, 64, 16000),
    ([1100], [1100], 4, 4, 64, 32, 1100),
    ([700, 3, 90, 1], [6000, 5, 20, 1], 4, 2, 128, 1024, 6000),
    ([257, 70], [4097, 0], 6, 2, 64, 128, 4097),
    ([2, 129, 2, 600, 2], [3000, 129, 17, 2048, 2], 8, 8, 128, 64, 2048),
    ([90] * 20, list(range(100, 1100, 50)), 16, 4, 64, 32, 11500),
]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("q_len,k_len,hq,hk,d,page,tokens", SHAPES)
def test_prompts_read_back(q_len, k_len, hq, hk, d, page, tokens, strided):
    """Runs of prompts with single tokens, drafts and segments without queries before, between and behind them."""
    g = gen(d + hq + page)
    cache, table = make(k_len, page, hk, d, ks=0.5, vs=4.0)
    fill(cache, table, k_len, BF, g)
    rows = sum(q_len) + 2
    q = randn((rows, hq + 3, d + 16), BF, g)[:, 1:1 + hq, :d] if strided else randn((rows, hq, d), BF, g)
    lse = torch.full((rows, hq), 7.0, device="cuda")
    buf = torch.full((rows, hq + 1, d), 7.0, dtype=BF, device="cuda")
    out = buf[:, :hq] if strided else buf[:, :hq].contiguous()
    assert rows_read_back(cache, q, table, q_len, k_len, tokens)
    cache.attend(q, table, q_len, k_len, out=out, lse=lse)
    check(q, *held(cache, table, k_len), q_len, k_len, d ** -0.5, out, lse)
    assert bool((out[-2:] == 7).all()) and bool((lse[-2:] == 7).all()) and bool((buf[:, hq:] == 7).all())
    ok()


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_over_their_queries_and_on_another_stream(d):
    g, q_len, k_len = gen(3), [1, 300, 2, 260], [700, 3000, 50, 260]
    cache, table = make(k_len, 64, 2, d)
    fill(cache, table, k_len, BF, g)
    q = randn((sum(q_len), 10, d), BF, g)[:, 1:-1]
    assert rows_read_back(cache, q, table, q_len, k_len, 3000)
    want = cache.attend(q, table, q_len, k_len)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = cache.attend(q, table, q_len, k_len, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert cache.attend(q, table, q_len, k_len, out=q) is q and torch.equal(q, want)
    ok()


def test_prompts_in_a_graph():
    g, q_len, k_len, d = gen(5), [1, 200, 150], [900, 4000, 300], 128
    cache, table = make(k_len, 64, 2, d)
    fill(cache, table, k_len, BF, g)
    q = randn((sum(q_len), 8, d), BF, g)
    space = torch.empty(cache.workspace(q, table, q_len, k_len), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q, table, q_len, k_len, out=out, lse=lse, workspace=space)
    for i in range(3):
        q.copy_(randn(q.shape, BF, g))
        graph.replay()
        want_lse = torch.empty_like(lse)
        want = cache.attend(q, table, q_len, k_len, lse=want_lse)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check(q, *held(cache, table, k_len), q_len, k_len, d ** -0.5, out, lse)
    ok()


FIRST = """
import sys; sys.path.insert(0, {root!r})
import torch
from heterogeneous_compressed_kv_gb300 import kvpool as K
n = 6000
cache = K.Kv4Cache(torch.zeros((100, K.kv4_page_bytes(2, 64, 64)), dtype=torch.uint8, device="cuda"), 2, 64, 64)
table = torch.arange(100, dtype=torch.int32, device="cuda")[None]
k = torch.randn((n, 2, 64), device="cuda").bfloat16()
q = torch.randn((300, 8, 64), device="cuda").bfloat16()
out = torch.zeros_like(q)
def call():
    cache.store(k, k, table, [0], [n])
    cache.attend(q, table, [300], [n], out=out)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
first = out.clone()
assert float(first.float().abs().sum()) > 0
call()
torch.cuda.synchronize()
assert torch.equal(first, out) and cache.workspace(q, table, [300], [n]) >= n * 2 * 64 * 4
assert K.window_check() == (K.OK, 0)
"""


def test_the_first_prompt_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_nan_in_a_prompt():
    """A NaN key reaches the queries that see it; places behind the tokens hold NaN scales (make fills pages with them)."""
    g, n, T, d = gen(7), 300, 5000, 64
    cache, table = make([T], 64, 1, d)
    k, v = randn((T, 1, d), BF, g), randn((T, 1, d), BF, g)
    k[T - 100, 0, 3] = math.nan
    cache.store(k, v, table, [0], [T])
    q, lse = randn((n, 8, d), BF, g), torch.empty((n, 8), device="cuda")
    q[5, 2, 7] = math.nan
    assert rows_read_back(cache, q, table, [n], [T], T)
    out = cache.attend(q, table, [n], [T], lse=lse)
    bad = torch.zeros((n, 8), dtype=torch.bool, device="cuda")
    bad[n - 100:], bad[5, 2] = True, True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad) and torch.equal(lse.isnan(), bad)
    ok()


# The kernel of single tokens has prompts as well: bf16 ones too short to be read back, held to its own bounds.
@pytest.mark.parametrize("q_len,k_len,hq,hk,d,page", [([70], [70], 1, 1, 64, 32), ([40, 1, 90], [200, 300, 111], 4, 2, 128, 32),
                                                      ([1, 80, 0, 65, 1], [9, 80, 7, 400, 100], 2, 1, 64, 32),
                                                      ([80, 100], [20, 0], 1, 1, 128, 32), ([200], [200], 4, 1, 64, 16),
                                                      ([33, 1, 150], [40, 900, 333], 4, 2, 128, 16), ([300], [1500], 2, 2, 64, 128)])
def test_prompts_of_the_small_products(q_len, k_len, hq, hk, d, page):
    from tests import test_gpu_kv4 as T
    g = gen(page + d)
    cache, table = make(k_len, page, hk, d)
    k, v = fill(cache, table, k_len, BF, g)
    q, lse = randn((sum(q_len), hq, d), BF, g), torch.empty((sum(q_len), hq), device="cuda")
    out = cache.attend(q, table, q_len, k_len, lse=lse)
    T.check(q, k, v, q_len, k_len, d ** -0.5, BF, out, lse)  # (weights in fp16: not the bounds of what is read back)
    ok()
