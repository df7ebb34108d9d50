"""Rows of a query tile that hold no query: with a group that does not divide 128 the last rows of a tile are nobody's."""
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("group,d", [(3, 128), (5, 64), (6, 128), (7, 64), (9, 128), (12, 64), (15, 128)])
def test_the_same_bits_whatever_ran_before(group, d):
    """A call's bits do not depend on what an earlier kernel left in shared memory: between two calls another one fills
    every row of its query tiles with large or with small values."""
    g = torch.Generator(device="cuda").manual_seed(group)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    n, T, hk = 500, 6000, 8
    size = 1 + torch.arange(T, device="cuda") / 1000  # later keys are larger: maxima keep growing
    k, v = (randn(T, hk, d) * size[:, None, None]).to(BF), randn(T, hk, d).to(BF)
    q = randn(n, hk * group, d).to(BF)
    fill = randn(2048, 16, d)
    runs = []
    for scale in (1e-3, 30.0, 1.0, 200.0):
        for heads in (16, 1):
            other = (fill * scale).to(BF)
            K.window_attend(other, other[:, :heads].contiguous(), other[:, :heads].contiguous(), [2048], [0], [2048], 1 << 20)
            lse = torch.empty((n, hk * group), device="cuda")
            runs.append((K.window_attend(q, k, v, [n], [0], [T], 1 << 20, lse=lse), lse))
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    assert K.window_check() == (K.OK, 0)


@pytest.mark.parametrize("group,d,n", [(1, 128, 130), (2, 64, 70), (4, 128, 33), (3, 64, 50)])
def test_the_same_bits_whatever_lies_behind_a_segment(group, d, n):
    """A query tile that ends inside the next segments' rows: a segment's bits do not depend on those, which outputs written
    over the queries may have replaced by then."""
    g = torch.Generator(device="cuda").manual_seed(group)
    segs, T, hk = 80, 2000, 8
    size = 1 + torch.arange(T, device="cuda") / 300  # later keys are larger: maxima keep growing
    k = (torch.randn((T, hk, d), device="cuda", generator=g) * size[:, None, None]).to(BF)
    v = torch.randn((T, hk, d), device="cuda", generator=g).to(BF)
    q = torch.randn((segs * n, hk * group, d), device="cuda", generator=g).to(BF)
    args = ([n] * segs, [0] * segs, [T] * segs, 1 << 20)
    want = K.window_attend(q, k, v, *args)
    for _ in range(3):
        over = q.clone()
        K.window_attend(over, k, v, *args, out=over)
        assert torch.equal(over, want)
    q.view(segs, n, hk * group, d)[1::2] *= 40  # every other segment's queries
    again = K.window_attend(q, k, v, *args)
    assert torch.equal(again.view(segs, -1)[0::2], want.view(segs, -1)[0::2])
    assert K.window_check() == (K.OK, 0)
