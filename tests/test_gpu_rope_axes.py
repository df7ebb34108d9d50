"""Rotation by positions of several axes against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests import test_gpu_rope as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def formula(x, pos, freq, axes, w, eps, inter):
    """R.formula with a position for each pair: every pair alone, by its axis."""
    out, mag = R.formula(x, torch.zeros_like(pos[:, 0]), freq, w, eps, inter)
    for a in set(axes):
        o, m = R.formula(x, pos[:, a], freq, w, eps, inter)
        rot = 2 * len(freq)
        for i in [i for i, b in enumerate(axes) if b == a]:
            for d in ((2 * i, 2 * i + 1) if inter else (i, i + rot // 2)):
                out[..., d], mag[..., d] = o[..., d], m[..., d]
    return out, mag


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,split", [(1, 1, 1, 64, 64, (8, 12, 12)), (37, 16, 4, 128, 128, (16, 24, 24)),
                                                 (700, 4, 1, 128, 64, (1, 0, 31)), (5, 3, 2, 256, 256, (16,) * 8),
                                                 (9, 2, 2, 96, 32, (16,)), (3, 5, 1, 80, 16, (4, 4))])
def test_formula(T, hq, hk, d, rot, split, inter, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    q, k = (torch.randn((T, h, d), device="cuda", generator=g).to(dtype) for h in (hq, hk))
    pos = torch.randint(-1000, 1 << 20, (T, len(split)), device="cuda", generator=g)
    axes = [a for a, n in enumerate(split) for _ in range(n)]
    np.random.RandomState(T).shuffle(axes)
    w = 1 + 0.2 * torch.randn((d,), device="cuda", generator=g)
    got = K.qk_norm_rope(q, k, pos, K.rope_table(rot), w, None, interleaved=inter, axes=axes)
    R.check(got[0], formula(q, pos, R.freqs(rot), axes, w, 1e-6, inter))
    R.check(got[1], formula(k, pos, R.freqs(rot), axes, None, 1e-6, inter))


def test_equal_positions_are_one_axis():
    """Text tokens have one position on every axis: the same bits as without axes; in place, as an array or a tensor of axes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((50, 8, 128), device="cuda", generator=g).bfloat16()
    pos, tab = torch.arange(50, device="cuda"), K.rope_table(128)
    axes = np.array([0] * 16 + [1] * 24 + [2] * 24)
    want = K.qk_norm_rope(q, None, pos, tab)[0]
    three = pos[:, None].expand(50, 3).contiguous()
    for a in (axes, torch.from_numpy(axes), axes.tolist(), bytes(axes.tolist())):
        assert torch.equal(K.qk_norm_rope(q, None, three, tab, axes=a)[0], want)
    assert torch.equal(K.qk_norm_rope(q, None, pos[:, None], tab, axes=[0] * 64)[0], want)
    assert K.qk_norm_rope(q, None, three, tab, axes=axes, out_q=q)[0] is q and torch.equal(q, want)


def test_refusals():
    q = torch.randn((4, 2, 64), device="cuda")
    pos, tab = torch.zeros((4, 3), dtype=torch.int64, device="cuda"), K.rope_table(64)
    good = [0] * 8 + [1] * 12 + [2] * 12
    K.qk_norm_rope(q, None, pos, tab, axes=good)
    for bad in (good[:-1], good + [0], [0.5] * 32, [-1] * 32, [300] * 32, 32, [good]):
        with pytest.raises(ValueError):
            K.qk_norm_rope(q, None, pos, tab, axes=bad)
    with pytest.raises(K.KvpoolError):
        K.qk_norm_rope(q, None, pos, tab, axes=[3] * 32)
    with pytest.raises(K.KvpoolError):
        K.qk_norm_rope(q, None, pos.repeat(1, 3), tab, axes=good)
    for p in (pos[:, 0], pos[:3], pos.float(), pos.t()):
        with pytest.raises(ValueError):
            K.qk_norm_rope(q, None, p, tab, axes=good)
    with pytest.raises(ValueError):
        K.qk_norm_rope(q, None, pos, tab)
    with pytest.raises(ValueError):
        K.qk_norm_rope(q, None, None, None, axes=good)
