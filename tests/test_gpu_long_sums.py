"""Prompts behind a million tokens: a sum of outputs over so many keys is not cut off step by step."""
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests.test_gpu_kv4 import gen, make
from tests.test_gpu_kv4_prompts import rows64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(n, T, hq, hk, d, g):
    """Values of one sign, of another size in every dim: a sum that loses a little of each addition loses it everywhere."""
    k = (0.3 * torch.randn((T, hk, d), device="cuda", generator=g)).to(BF)
    v = torch.randn((T, hk, d), device="cuda", generator=g).abs_()
    v = (v * (1 + torch.rand((hk, d), device="cuda", generator=g))).to(BF)
    return torch.randn((n, hq, d), device="cuda", generator=g).to(BF), k, v


def close(out, q, k, v, n, T):
    """The mean relative error of the last 16 queries' outputs.  What the outputs' rounding (2^-8 of each at most, of no sign)
    leaves of it in hq * d places of unlike sizes, 16 times the same ones: 2^-8 / sqrt(3) / sqrt(hq * d) = 2^-13.3 at 512,
    three times that 2^-11.7; the weights' rounding, over a million of them, 2^-17.  A sum over 16,384 keys loses 2^-23 of
    itself in each of 1,024 additions at most: 2^-13.  Together less than 2^-11."""
    o = rows64(q[n - 16:], torch.arange(T - 16, T, device="cuda"), k, v, q.shape[2] ** -0.5)[0]
    assert abs(float(((out[n - 16:].double() - o) / o).mean())) < 2.0 ** -11


@pytest.mark.parametrize("n,T,hq,hk,d", [(4096, 1 << 20, 16, 4, 128), (1024, 1 << 20, 16, 4, 128), (8192, 600_001, 8, 8, 64), (600, 1 << 20, 12, 4, 128)])
def test_prompts_over_the_4_bit_cache(n, T, hq, hk, d):
    q, k, v = inputs(n, T, hq, hk, d, gen(n))
    cache, table = make([T], 256, hk, d)
    cache.store(k, v, table, [0], [T])
    out = cache.attend(q, table, [n], [T])
    k, v = cache.load(table, [0], [T], dtype=F32)
    close(out, q, k.double(), v.double(), n, T)
    assert K.window_check() == (K.OK, 0)


@pytest.mark.parametrize("n,T,hq,hk,d,window", [(2500, 1 << 20, 16, 4, 128, 1 << 20), (2500, 1 << 20, 16, 4, 128, 500_000), (5000, 600_001, 8, 8, 64, 1 << 22)])
def test_window_attention(n, T, hq, hk, d, window):
    q, k, v = inputs(n, T, hq, hk, d, gen(n + 1))
    want = torch.full((n + 1, hq), 7.0, device="cuda")
    out = K.window_attend(q, k, v, [n], [0], [T], window, lse=want[:-1])
    lo = max(0, T - 15 - window)  # (what the last 16 queries see differs by a few keys of many: they are cut alike)
    if lo == 0:
        close(out, q, k.double(), v.double(), n, T)
    else:
        q16 = q[n - 1:].double()
        for h in range(hq):
            kh, vh = k[T - window:, h // (hq // hk)].double(), v[T - window:, h // (hq // hk)].double()
            p = torch.softmax(q16[:, h] @ kh.T * d ** -0.5, -1)
            if h == 0:
                err = []
            err.append(((out[n - 1:, h].double() - p @ vh) / (p @ vh)).mean())
        assert abs(float(torch.stack(err).mean())) < 2.0 ** -11
    assert K.window_check() == (K.OK, 0)
    # queries over themselves, and in a second call: the same bits
    again = K.window_attend(q, k, v, [n], [0], [T], window)
    assert torch.equal(again, out) and torch.equal(K.window_attend(q, k, v, [n], [0], [T], window, out=q), out)


@pytest.mark.parametrize("n,T,hq,hk,d,q_len", [(160, 1 << 20, 16, 4, 128, 1), (200, 700_003, 8, 8, 64, 2)])
def test_single_tokens_and_drafts(n, T, hq, hk, d, q_len):
    """More requests than the GPU holds work items of, all behind the same rows: no request's keys are cut for the GPU's sake."""
    q, k, v = inputs(n * q_len, T, hq, hk, d, gen(n))
    out = K.window_attend(q, k, v, [q_len] * n, [0] * n, [T] * n, 1 << 20)
    last = out.view(n, q_len, hq, d)[:16, -1].contiguous()  # (the last query of 16 requests sees all)
    o = rows64(q.view(n, q_len, hq, d)[:16, -1], torch.full((16,), T - 1, device="cuda"), k.double(), v.double(), d ** -0.5)[0]
    assert abs(float(((last.double() - o) / o).mean())) < 2.0 ** -11
    assert K.window_check() == (K.OK, 0)


@pytest.mark.parametrize("n,T,hq,hk,d,q_len", [(500, 1 << 20, 16, 4, 128, 1), (1500, 1 << 20, 8, 2, 128, 1), (900, 700_003, 8, 4, 128, 2)])
def test_single_tokens_over_the_4_bit_cache(n, T, hq, hk, d, q_len):
    """Requests that share their pages, so many that every warp of the GPU has more than a unit's keys of them."""
    q, k, v = inputs(n * q_len, T, hq, hk, d, gen(n))
    cache, table = make([T], 256, hk, d)
    cache.store(k, v, table, [0], [T])
    out = cache.attend(q, table.expand(n, table.shape[1]), [q_len] * n, [T] * n)
    k, v = cache.load(table, [0], [T], dtype=F32)
    at = slice(n // 2, n // 2 + 16)
    last = out.view(n, q_len, hq, d)[at, -1]
    o = rows64(q.view(n, q_len, hq, d)[at, -1].contiguous(), torch.full((16,), T - 1, device="cuda"), k.double(), v.double(), d ** -0.5)[0]
    assert abs(float(((last.double() - o) / o).mean())) < 2.0 ** -11
    assert K.window_check() == (K.OK, 0)


def test_weights_where_shares_take_several_rounds():
    n, T, h, d = 160, 1 << 20, 4, 128
    q, k, v = inputs(n, T, h, h, d, gen(7))
    cache, table = make([T], 256, h, d)
    cache.store(k, v, table, [0], [T])
    k = cache.load(table, [0], [T], dtype=F32)[0].double()
    w, lse = torch.full((n, h, T), 3.0, device="cuda"), torch.empty((n, h), device="cuda")
    cache.attend(q, table.expand(n, table.shape[1]), [1] * n, [T] * n, lse=lse, weights=w, decay=0.5)
    for i in (0, 77, 159):
        for j in range(h):
            s = q[i, j].double() @ k[:, j].T * d ** -0.5
            z = torch.logsumexp(s, -1)
            assert float((lse[i, j] - z).abs()) < 1e-5  # (2^-17 of sums of |q k|, about 0.3)
            # a half step of numbers from 1 to 2, and 2^-17 of weights that are below 1e-4
            assert float((w[i, j].double() - 1.5 - torch.exp(s - z)).abs().max()) < 2.0 ** -23
    assert K.window_check() == (K.OK, 0)


@pytest.mark.parametrize("n,T,hk,group,d,window,sink", [
    (600, 90_001, 2, 3, 64, 33_000, 17_001), (2500, 60_000, 1, 4, 128, 17_000, 40_000), (2500, 90_001, 4, 8, 64, 1 << 20, 130),
    (300, 40_000, 4, 2, 128, 20_000, 3), (1, 90_001, 2, 8, 128, 70_000, 17_001), (3, 200_003, 1, 1, 64, 1 << 20, 0)])
def test_first_tokens_before_long_windows(n, T, hk, group, d, window, sink):
    """Steps over the first tokens and over the window in one item, against 64 bits: weights are rounded to 2^-8 of each,
    outputs once more, scores are off by less than 1e-4 (2^-17 of sums of |q k| scale, below 10)."""
    g = gen(T + n)
    q, k, v = (torch.randn(s, device="cuda", generator=g).to(BF) for s in ((n, hk * group, d), (T, hk, d), (T, hk, d)))
    lse = torch.empty((n, hk * group), device="cuda")
    out = K.window_attend(q, k, v, [n], [0], [T], window, sink, lse=lse)
    j = torch.unique(torch.tensor([0, n // 3, n // 2, n - 2, n - 1], device="cuda").clamp(0))
    pos, t = T - n + j, torch.arange(T, device="cuda")
    hidden = ~((t[None] <= pos[:, None]) & ((t[None] > pos[:, None] - window) | (t[None] < sink)))
    for h in range(hk * group):
        s = (q[j, h].double() @ k[:, h // group].double().T * d ** -0.5).masked_fill(hidden, -float("inf"))
        z = torch.logsumexp(s, -1)
        p, x = torch.exp(s - z[:, None]), v[:, h // group].double()
        o = p @ x
        assert bool(((out[j, h].double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 3e-4) * (p @ x.abs()) + 1e-9).all())
        assert float((lse[j, h] - z).abs().max()) < 1e-4
    over = q.clone()
    assert torch.equal(K.window_attend(over, k, v, [n], [0], [T], window, sink, out=over), out)
    assert K.window_check() == (K.OK, 0)
