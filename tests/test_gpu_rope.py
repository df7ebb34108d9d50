"""Head norms with the position rotation against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K

pytestmark = pytest.mark.gpu


def formula(x, pos, freq, w, eps, inter):
    """The rotated norms in 64 bits, and each value's pair magnitude."""
    x = x.double().cpu()
    rot = 2 * len(freq)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double().cpu()
    ang = pos.double().cpu()[:, None, None] * torch.tensor(freq, dtype=torch.float64)
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    p, q = a * torch.cos(ang) - b * torch.sin(ang), b * torch.cos(ang) + a * torch.sin(ang)
    mag = torch.sqrt(a * a + b * b)
    if inter:
        r, g = torch.stack([p, q], -1).flatten(-2), torch.stack([mag, mag], -1).flatten(-2)
    else:
        r, g = torch.cat([p, q], -1), torch.cat([mag, mag], -1)
    return torch.cat([r, y[..., rot:]], -1), torch.cat([g, y[..., rot:].abs()], -1)


def check(got, want):
    ref, mag = want
    # one rounding to the type (half a step of the value), and in fp32: the sum of squares and its root (a few steps),
    # the sine's and cosine's place (2^-25 turns, 2 pi of it: 2^-22.3) and two products: under 2^-20 of the pair
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + 2.0 ** -20 * mag + 1e-30
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def freqs(rot):
    return 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot", [(1, 1, 1, 64, 64), (3, 4, 1, 128, 128), (33, 16, 16, 128, 64), (5, 3, 2, 96, 32),
                                           (7, 5, 1, 256, 256), (2, 2, 2, 8, 0), (4, 9, 3, 80, 80), (700, 16, 2, 64, 48),
                                           (3000, 16, 4, 128, 128)])
def test_formula(T, hq, hk, d, rot, inter, dtype):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + d)
    q = torch.randn((T, hq, d), device="cuda", generator=g).to(dtype)
    k = (3 * torch.randn((T, hk, d), device="cuda", generator=g)).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", generator=g)
    qw = torch.randn((d,), device="cuda", generator=g)
    tab = K.rope_table(rot) if rot else None
    oq, ok = K.qk_norm_rope(q, k, pos, tab, qw, None, eps=1e-5, interleaved=inter)
    check(oq, formula(q, pos, freqs(rot), qw, 1e-5, inter))
    check(ok, formula(k, pos, freqs(rot), None, 1e-5, inter))


def test_far_and_negative_positions():
    # the turn is exact modulo 2^64, so a position far away is as good as a near one; the formula's own angle in 64 bits
    # is good to 2^-53 of itself, which holds 2^20 radians to 2^-33
    pos = torch.tensor([0, 1, -1, 1 << 20, -(1 << 20), (1 << 20) + 1], device="cuda")
    q = torch.randn((6, 2, 128), device="cuda")
    oq, _ = K.qk_norm_rope(q, None, pos, K.rope_table(128))
    check(oq, formula(q, pos, freqs(128), None, 1e-6, False))
    # exact periods: a frequency of a quarter turn comes back after 4 positions, at any distance
    tab = K.rope_table(16, inv_freq=np.full(8, np.pi / 2))
    far = torch.tensor([0, 4, 1 << 40, -(1 << 40), (1 << 62) + 4, 2], device="cuda")
    x = torch.randn((1, 1, 16), device="cuda").expand(6, 1, 16).contiguous()
    y, _ = K.qk_norm_rope(x, None, far, tab)
    for i in range(1, 5):
        assert torch.equal(y[0], y[i])
    assert torch.equal(y[5], -y[0])


def test_zeros_and_extremes():
    x = torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16)
    pos = torch.tensor([0, 5], device="cuda")
    y, _ = K.qk_norm_rope(x, None, pos, K.rope_table(64))
    assert torch.equal(y, x)
    big = torch.full((1, 1, 64), 1e18, device="cuda")
    y, _ = K.qk_norm_rope(big, None, pos[:1], K.rope_table(64))  # squares of 1e36 still sum in fp32
    check(y, formula(big, pos[:1], freqs(64), None, 1e-6, False))


def test_views_in_place_and_rows_behind():
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn((9, 8 + 2 * 2, 128), device="cuda", generator=g).bfloat16()
    keep = rows.clone()
    pos = torch.arange(100, 107, device="cuda")
    tab = K.rope_table(128)
    q, k = rows[:7, :8], rows[:7, 8:10]
    wq, wk = K.qk_norm_rope(q, k, pos, tab)
    oq, ok = K.qk_norm_rope(q, k, pos, tab, out_q=q, out_k=k)  # in place, inside a fused projection's rows
    assert oq.data_ptr() == q.data_ptr() and torch.equal(oq, wq) and torch.equal(ok, wk)
    assert torch.equal(rows[:, 10:], keep[:, 10:]) and torch.equal(rows[7:], keep[7:])
    # heads outermost
    x = torch.randn((4, 7, 64), device="cuda", generator=g).transpose(0, 1)
    y, _ = K.qk_norm_rope(x, None, pos, K.rope_table(64))
    check(y, formula(x, pos, freqs(64), None, 1e-6, False))


def test_no_tokens():
    q = torch.empty((0, 4, 64), device="cuda", dtype=torch.bfloat16)
    oq, ok = K.qk_norm_rope(q, None, torch.empty((0,), dtype=torch.int64, device="cuda"), K.rope_table(64))
    assert oq.shape == q.shape and ok is None


def test_refusals():
    q = torch.randn((4, 2, 64), device="cuda")
    pos, tab = torch.arange(4, device="cuda"), K.rope_table(64)
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[:, :, ::2]), dict(q=torch.randn((4, 2, 66), device="cuda")[:, :, 1:65]),
                dict(positions=pos.int()), dict(positions=pos[:3]), dict(table=tab.float()), dict(q_weight=pos),
                dict(k=q.bfloat16()), dict(k=q[:3]), dict(out_q=q[:3]), dict(out_q=q[:, :1].expand(4, 2, 64))):
        with pytest.raises(ValueError):
            K.qk_norm_rope(**{**dict(q=q, k=None, positions=pos, table=tab), **bad})
    with pytest.raises(K.KvpoolError):
        K.qk_norm_rope(q, None, pos, K.rope_table(128))  # rot_dim above head_dim
    with pytest.raises(ValueError):
        K.qk_norm_rope(None, None, pos, tab)


def test_stream_and_graph():
    q = torch.randn((40, 16, 128), device="cuda").bfloat16()
    pos, tab = torch.arange(40, device="cuda"), K.rope_table(128)
    want, _ = K.qk_norm_rope(q, None, pos, tab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = K.qk_norm_rope(q, None, pos, tab, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.qk_norm_rope(q, None, pos, tab, out_q=out)
    pos += 11
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, K.qk_norm_rope(q, None, pos, tab)[0])


def test_outputs_whose_heads_lie_on_each_other_are_refused():
    q = torch.randn((4, 2, 64), device="cuda")
    pos, tab = torch.arange(4, device="cuda"), K.rope_table(64)
    space = torch.zeros(64 * 16, device="cuda")
    on_each_other = torch.as_strided(space, (4, 2, 64), (64, 64, 1))  # head 1 of a token on head 0 of the next
    with pytest.raises(ValueError):
        K.qk_norm_rope(q, None, pos, tab, out_q=on_each_other)
    with pytest.raises(ValueError):
        K.window_attend(q, q, q, [4], [0], [4], 4, out=on_each_other)
    assert bool((space == 0).all())
    want, _ = K.qk_norm_rope(q, None, pos, tab)
    for strides in ((192, 72, 1), (72, 288, 1)):  # heads within a token, tokens within a head, with room in between
        o = torch.as_strided(space, (4, 2, 64), strides)
        got, _ = K.qk_norm_rope(q, None, pos, tab, out_q=o)
        assert got.data_ptr() == o.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 2, 5])
def test_outputs_among_the_inputs_rows(T):
    """The layouts of one buffer that lie apart, or in place, give what an output of its own gives; all others are refused
    and write nothing."""
    from tests.test_ops_host import FUSED, P16, meets
    g = torch.Generator(device="cuda").manual_seed(4)
    pos, tab = torch.arange(T, device="cuda") + 3, K.rope_table(64)
    for layout in FUSED:
        space = torch.randn((4096,), device="cuda", generator=g).bfloat16()
        keep = space.clone()
        q, k, o = (torch.as_strided(space, (T, n, 64), (ts, hs, 1), (p - P16) // 2) for p, ts, hs, n, _ in layout)
        wq, wk = K.qk_norm_rope(q.clone(), k.clone(), pos, tab)
        ww = K.window_attend(q.clone(), k.clone(), k.clone(), [T], [0], [T], 16)
        if meets(*layout, T):
            with pytest.raises(K.KvpoolError):
                K.qk_norm_rope(q, k, pos, tab, out_q=o)
            with pytest.raises(K.KvpoolError):
                K.window_attend(q, k, k, [T], [0], [T], 16, out=o)
            assert torch.equal(space, keep)
            continue
        lk = k.clone()
        oq, ok = K.qk_norm_rope(q, k, pos, tab, out_q=o)
        assert torch.equal(oq, wq) and torch.equal(ok, wk) and torch.equal(k, lk)
        space.copy_(keep)
        assert torch.equal(K.window_attend(q, k, k, [T], [0], [T], 16, out=o), ww) and torch.equal(k, lk)


@pytest.mark.parametrize("ql,kl,window,dtype,scale", [
    ([1, 3], [40, 300], 64, torch.bfloat16, None), ([1], [9000], 8000, torch.bfloat16, None), ([2], [9000], 8000, torch.float32, None),
    ([70, 300, 1], [100, 500, 90], 128, torch.bfloat16, None), ([40], [5000], 4096, torch.bfloat16, None),
    ([70, 300], [100, 500], 128, torch.float32, None), ([70, 300], [100, 500], 128, torch.bfloat16, -0.1)])
def test_window_outputs_in_the_queries_place(ql, kl, window, dtype, scale):
    g = torch.Generator(device="cuda").manual_seed(sum(kl))
    rows = torch.randn((sum(ql), 6 + 2, 64), device="cuda", generator=g).to(dtype)
    k, v = (torch.randn((sum(kl), 2, 64), device="cuda", generator=g).to(dtype) for _ in range(2))
    ks = [0] + list(np.cumsum(kl)[:-1])
    keep, q = rows.clone(), rows[:, :6]
    want = K.window_attend(q, k, v, ql, ks, kl, window, 2, scale=scale)
    got = K.window_attend(q, k, v, ql, ks, kl, window, 2, scale=scale, out=q)
    assert got.data_ptr() == rows.data_ptr() and torch.equal(got, want) and torch.equal(rows[:, 6:], keep[:, 6:])


def exact_turns(p, f):
    """The fraction of a turn of angle p f, from integers: pi to 400 bits by Machin's formula."""
    from fractions import Fraction
    one = 1 << 400

    def arctan_inv(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    two_pi = Fraction(2 * 4 * (4 * arctan_inv(5) - arctan_inv(239)), one)
    t = Fraction(int(p)) * Fraction(float(f)) / two_pi
    return float(t - (t.numerator // t.denominator)), abs(float(t))


@pytest.mark.parametrize("p", [1 << 20, 1 << 31, 1 << 40, -(1 << 40) - 12345, 1 << 50])
def test_angles_of_far_positions_hold_what_is_said_of_them(p):
    """Frequencies of no particular relation to a turn: 2^-25 turns, 2^-52 of the turns and p 2^-64 (cosine and sine move
    by 2 pi times that at most), and fp32 arithmetic as in check().  The last of the three: a table entry is cut off at
    2^-64, so it is short of the quotient by less than that, and p of them by less than p 2^-64."""
    f = np.array([1.0, 0.7316, 10000 ** -0.25, 0.1, 3.3, 2.0 ** -9 * 1.37, 1e-4, 17.77])
    x = torch.randn((1, 3, 16), device="cuda")
    y, _ = K.qk_norm_rope(x, None, torch.tensor([p], device="cuda"), K.rope_table(16, inv_freq=f))
    turns, count = (torch.tensor(z, dtype=torch.float64) for z in zip(*(exact_turns(p, v) for v in f)))
    n = x.double().cpu()
    n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + 1e-6)
    a, b = n[..., :8], n[..., 8:]
    c, s = torch.cos(2 * np.pi * turns), torch.sin(2 * np.pi * turns)
    mag = torch.cat([torch.sqrt(a * a + b * b)] * 2, -1)
    want = torch.cat([a * c - b * s, b * c + a * s], -1)
    tol = (2.0 ** -20 + 2 * np.pi * (2.0 ** -25 + count * 2.0 ** -52 + abs(p) * 2.0 ** -64)).repeat(2) * mag
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
