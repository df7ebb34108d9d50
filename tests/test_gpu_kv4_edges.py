"""The 4-bit paged cache at the edges of what its calls allow."""
import math

import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests import kv4_format as F
from tests.test_gpu_kv4 import BF, F32, fill, gen, make, ok, randn, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", ["negative", "zero", "heads alike", "tokens alike"])
def test_prompts_that_the_tensor_copies_cannot_take(case):
    """Long bf16 segments whose scale or strides window attention's tensor-core form does not take stay where they are
    quick: nothing is read back, and the answers are those of the formula."""
    from tests.test_gpu_kv4_prompts import check, held
    g, n, T, hq, hk, d = gen(17), 300, 6000, 8, 2, 64
    cache, table = make([T], 64, hk, d)
    fill(cache, table, [T], BF, g)
    q = randn((n, hq, d), BF, g)
    scale = {"negative": -0.125, "zero": 0.0}.get(case, 0.125)
    if case == "heads alike":
        q = q[:, :1].expand(n, hq, d)
    if case == "tokens alike":
        q = q[:1].expand(n, hq, d)
    assert cache.workspace(q, table, [n], [T], scale=scale) < T * hk * d * 4
    out, lse = torch.empty((n, hq, d), dtype=BF, device="cuda"), torch.empty((n, hq), device="cuda")
    cache.attend(q, table, [n], [T], scale=scale, out=out, lse=lse)
    check(q, *held(cache, table, [T]), [n], [T], scale, out, lse)
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("q_len,k_len,hq,hk,d,weigh", [
    (1, 1, 4, 1, 64, True), (1, 1, 1, 1, 128, False), (3, 40, 4, 2, 128, True), (1, 9000, 8, 1, 64, True), (4, 3, 2, 1, 64, True),
    (5, 9000, 16, 1, 128, False), (100, 300, 2, 1, 64, False), (300, 4000, 8, 2, 128, False), (310, 300, 8, 8, 64, False)])
def test_infinite_queries(q_len, k_len, hq, hk, d, weigh, sign, dtype):
    """A query that is infinite in a dim in which every key has the same sign gives NaN, and no other query does; one that
    sees no token gives zeros."""
    g = gen(q_len + k_len)
    cache, table = make([k_len], 32, hk, d)
    k, v = randn((k_len, hk, d), dtype, g), randn((k_len, hk, d), dtype, g)
    k[..., 3] = k[..., 3].abs() + 4  # (no scale makes a zero of it)
    cache.store(k, v, table, [0], [k_len])
    q, lse = randn((q_len, hq, d), dtype, g), torch.empty((q_len, hq), device="cuda")
    w = torch.zeros((1, hk, k_len), device="cuda") if weigh else None
    at = sorted({0, q_len // 2, q_len - 1})
    for i, j in enumerate(at):
        q[j, (i + 1) % hq, 3] = sign * math.inf
    out = cache.attend(q, table, [q_len], [k_len], lse=lse, weights=w, decay=0.0)
    bad = torch.zeros((q_len, hq), dtype=torch.bool, device="cuda")
    nothing = max(0, q_len - k_len)
    for i, j in enumerate(at):
        bad[j, (i + 1) % hq] = j >= nothing
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad)
    assert bool((out[:nothing] == 0).all()) and bool((lse[:nothing] == -math.inf).all())
    if weigh:  # a row of NaN makes NaNs of its head's weights, and of no other's
        heads = bad.any(0).view(hk, -1).any(-1)
        assert torch.equal(w[0].isnan().all(-1), heads) and torch.equal(w[0].isnan().any(-1), heads)
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ks,vs", [(2.0 ** -16, 2.0 ** -3), (2.0 ** -12, 1.0), (1.0, 2.0 ** -16), (2.0 ** 16, 2.0 ** -16)])
def test_values_too_large_for_a_scale(ks, vs, dtype):
    """Finite values of any size are held as 2688 scales at most: where x / k_scale is past fp32's range as well."""
    x = torch.zeros((1, 1, 128))
    for i, big in enumerate((3e38, -1e35, 2e34, 1e30, 3e5, -3.3e38, 1.0, 1e-3)):
        x[0, 0, 16 * i:16 * i + 16] = torch.linspace(-1, 1, 16)
        x[0, 0, 16 * i + i] = big
        x[0, 0, 16 * i + 15 - i] = -big / 2
    x = x.to(dtype).cuda()
    cache, table = make([3], 16, 1, 128, ks=ks, vs=vs)
    cache.store(x, x, table, [1], [1])
    got = cache.load(table, [1], [1], dtype=F32)
    for y, s in zip(got, (ks, vs)):
        # what is past 2688 scales is held as that, so a smaller number past it has the same codes
        top = 2.0 ** 20 * s
        assert same(y, F.held(x.float().clamp(-top, top), s)) and not bool(y.isnan().any())
    ok()


def test_load_into_one_given_output():
    """Either output of load may be given, with rows behind the tokens."""
    g, T = gen(13), 40
    cache, table = make([T], 16, 2, 64)
    k, v = fill(cache, table, [T], BF, g)
    for dtype in (BF, F32):
        o = torch.full((T + 3, 2, 64), 9.0, dtype=dtype, device="cuda")
        a, b = cache.load(table, [0], [T], out_k=o)
        assert a is o and b.dtype is dtype and b.shape == o.shape and same(o[:T], k) and same(b[:T], v) and bool((o[T:] == 9).all())
        a, b = cache.load(table, [0], [T], out_v=o)
        assert b is o and a.dtype is dtype and same(o[:T], v) and same(a[:T], k) and bool((o[T:] == 9).all())
    with pytest.raises(ValueError):
        cache.load(table, [0], [T], dtype=BF, out_k=o)
    ok()


SPACE = 9 << 28  # bytes that a call without weights asks for at most


@pytest.mark.parametrize("q_len,k_len,hq,hk,d", [
    ([1024], [1 << 20], 16, 16, 128), ([5] * 64, [131072] * 64, 64, 4, 128), ([4096] * 4, [1 << 18] * 4, 64, 64, 128), ([2048], [1 << 24], 16, 1, 64),
    ([1 << 20], [1 << 20], 16, 4, 128), ([512], [1 << 16], 1024, 1024, 128), ([80] * 500, [40000] * 500, 8, 8, 64)])
def test_a_prompt_s_workspace_is_bounded(q_len, k_len, hq, hk, d):
    """However many tokens are read back, their rows do not lie in the workspace all at once.  (Sizes only.)"""
    cache = K.Kv4Cache(torch.zeros((1, K.kv4_page_bytes(hk, d, 1024)), dtype=torch.uint8, device="cuda"), hk, d, 1024)
    table = torch.zeros((len(k_len), max(k_len) // 1024 + 1), dtype=torch.int32, device="cuda")
    q = torch.empty((sum(q_len), hq, d), dtype=BF, device="cuda")
    assert cache.workspace(q, table, q_len, k_len) <= SPACE


@pytest.mark.parametrize("q_len,k_len,hq,hk,d,page", [
    ([40], [70001], 128, 64, 128, 64), ([1, 70, 200, 2], [300, 66000, 3000, 70], 256, 128, 64, 16),
    ([9001], [66003], 64, 64, 128, 1024), ([70100], [66010], 64, 64, 128, 256), ([300, 300], [65536, 131073], 64, 64, 128, 64),
    ([128], [100000], 192, 64, 128, 128)])
def test_prompts_behind_more_tokens_than_are_read_back_at_once(q_len, k_len, hq, hk, d, page):
    """Segments of more than 65,536 tokens at these heads are attended to a piece at a time (of queries too, where there are
    many), their running sums kept in between: beside others, over their own queries, and with an infinite query."""
    from tests.test_gpu_kv4_prompts import check, held
    g = gen(sum(q_len) + hk)
    cache, table = make(k_len, page, hk, d)
    fill_in_parts(cache, table, k_len, g)
    rows = sum(q_len) + 2
    buf = randn((rows, hq + 1, d), BF, g)
    q = buf[:, :hq]
    lse = torch.full((rows, hq), 7.0, device="cuda")
    out = torch.full((rows, hq, d), 7.0, dtype=BF, device="cuda")
    assert cache.workspace(q, table, q_len, k_len) <= SPACE
    cache.attend(q, table, q_len, k_len, out=out, lse=lse)
    k, v = held(cache, table, k_len)
    check(q, k, v, q_len, k_len, d ** -0.5, out, lse)
    assert bool((out[-2:] == 7).all()) and bool((lse[-2:] == 7).all())
    # An infinite query makes its own row NaN.  The rows of its warp may be rescaled at another step than before (one row's
    # larger maximum rescales them all), which moves their roundings: they are held to the formula again, not to the same bits.
    row, finite, want = sum(q_len) - 1, q.clone(), out.clone()
    q[row, 1, 0] = math.inf
    cache.attend(q, table, q_len, k_len, out=want)
    assert bool(want[row, 1].isnan().all())
    other = want.clone()
    other[row, 1] = out[row, 1]
    check(finite, k, v, q_len, k_len, d ** -0.5, other, lse)
    last, behind = buf[:, hq].clone(), q[-2:].clone()
    cache.attend(q, table, q_len, k_len, out=q)
    assert same(q[:-2], want[:-2]) and torch.equal(buf[:, hq], last) and torch.equal(q[-2:], behind)
    ok()


def fill_in_parts(cache, table, lens, g, v_size=1.0):
    for i, n in enumerate(lens):
        for t in range(0, n, 1 << 15):
            m = min(1 << 15, n - t)
            k, v = (randn((m, cache.kv_heads, cache.head_dim), BF, g) for _ in range(2))
            cache.store(k, v * v_size, table[i:i + 1], [t], [m])


@pytest.mark.parametrize("q_len,k_len,hq,hk,d,scale", [
    ([1, 300, 0, 200, 1, 150], [50, 4000, 30, 2500, 700, 150], 8, 2, 128, 1.0), ([100, 5], [8000, 8000], 16, 1, 64, 0.5),
    ([700], [6000], 6, 2, 64, 2.0), ([600], [60000], 4, 4, 128, None), ([128], [66000], 64, 64, 128, 0.3)])
def test_weights_of_prompts_that_are_read_back_have_eleven_bits(q_len, k_len, hq, hk, d, scale):
    """However a segment is attended to, softmax weights go into their products with half an fp16 step each (2^-11): scales
    that make a few of them large show it."""
    from tests.test_gpu_kv4_prompts import check, held, rows_read_back
    g = gen(hq + d)
    scale = d ** -0.5 if scale is None else scale
    cache, table = make(k_len, 64, hk, d, vs=2.0 ** -14)
    fill_in_parts(cache, table, k_len, g, 2.0 ** -14)
    q, lse = randn((sum(q_len), hq, d), BF, g), torch.empty((sum(q_len), hq), device="cuda")
    assert rows_read_back(cache, q, table, q_len, k_len, 2000, scale=scale)
    out = cache.attend(q, table, q_len, k_len, scale=scale, lse=lse)
    check(q, *held(cache, table, k_len), q_len, k_len, scale, out, lse, r=2.0 ** -11)
    ok()


def test_a_segment_in_pieces_in_a_graph():
    g, q_len, k_len = gen(9), [40, 5], [70000, 300]
    cache, table = make(k_len, 64, 64, 128)
    fill_in_parts(cache, table, k_len, g)
    q = randn((45, 128, 128), BF, g)
    out, space = torch.zeros_like(q), torch.empty(cache.workspace(q, table, q_len, k_len), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q, table, q_len, k_len, out=out, workspace=space)
    for _ in range(2):
        q.copy_(randn(q.shape, BF, g))
        graph.replay()
        assert torch.equal(out, cache.attend(q, table, q_len, k_len))
    ok()
