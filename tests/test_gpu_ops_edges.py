"""Calls around the pool that their documentation allows at the edges: rows further apart than 32 bits count, the first
call of a process inside a capture, two threads at once, the same call again bit for bit."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests import test_gpu_rope as R
from tests import test_gpu_window as Wn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("ql,kl,window,dtype,scale", [([1], [700], 300, BF, None), ([3], [700], 300, F32, None),
                                                      ([90], [700], 128, BF, None), ([90], [700], 128, F32, None),
                                                      ([90], [700], 128, BF, -0.1), ([40], [5000], 4096, BF, None)])
def test_window_rows_past_32_bits(ql, kl, window, dtype, scale):
    """Keys and values whose last rows are more than 2^32 values behind the first one, a segment at their end; queries
    and outputs likewise."""
    q, k, v, _ = Wn.inputs(ql, kl, 4, 2, 64, dtype)
    n, m, step = ql[0], kl[0], 1 << 17
    rows = (1 << 32) // step + m + 5
    space = torch.empty((rows + 1) * step, dtype=dtype, device="cuda")
    at = rows - m
    far = [torch.as_strided(space, (rows, 2, 64), (step, 64, 1), off) for off in (0, 1024)]
    for x, y in zip(far, (k, v)):
        x[at:] = y
    lse = torch.empty((n, 4), device="cuda")
    out = K.window_attend(q, *far, ql, [at], kl, window, 2, scale=scale, lse=lse)
    want = K.window_attend(q, k, v, ql, [0], kl, window, 2, scale=scale)
    assert torch.equal(out, want)
    # queries and outputs, one row each beyond 2^32 values from the next
    big = (1 << 32) // max(n - 1, 1) // 64 * 64 + 64
    if n > 1:
        qs, os_ = (torch.as_strided(space, (n, 4, 64), (big, 64, 1), off) for off in (2048, 4096))
        if (n - 1) * big + 8192 <= space.numel():
            qs.copy_(q)
            got = K.window_attend(qs, k, v, ql, [0], kl, window, 2, scale=scale, out=os_)
            assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotation_rows_past_32_bits(dtype):
    T, step = 5, (1 << 30) + 64
    space = torch.empty((T - 1) * step + 8192, dtype=dtype, device="cuda")
    q = torch.as_strided(space, (T, 3, 128), (step, 128, 1))
    k = torch.as_strided(space, (T, 1, 128), (step, 128, 1), 1024)
    g = torch.Generator(device="cuda").manual_seed(2)
    for x in (q, k):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
    pos, tab = torch.arange(T, device="cuda") * 1000, K.rope_table(128)
    want = [R.formula(x.clone(), pos, R.freqs(128), None, 1e-6, False) for x in (q, k)]
    for got, w in zip(K.qk_norm_rope(q, k, pos, tab, out_q=q, out_k=k), want):
        R.check(got, w)


FIRST = """
import sys; sys.path.insert(0, {root!r})
import torch
from heterogeneous_compressed_kv_gb300 import kvpool as K
q = torch.randn((300, 4, 64), device="cuda").bfloat16()
k = torch.randn((300, 2, 64), device="cuda").bfloat16()
pos, tab = torch.arange(300, device="cuda"), K.rope_table(64)
out, f = torch.zeros_like(q), {f32}
if f:
    q, k, out = q.float(), k.float(), out.float()
call = lambda: {call}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
first = out.clone()
assert float(first.float().abs().sum()) > 0
out.zero_()
call()
torch.cuda.synchronize()
assert torch.equal(first, out)
"""


@pytest.mark.parametrize("call,f32", [
    ("K.qk_norm_rope(q, None, pos, tab, out_q=out)", False),
    ("K.window_attend(q, k, k, [300], [0], [300], 100, 2, out=out)", False),
    ("K.window_attend(q, k, k, [300], [0], [300], 100, 2, out=out)", True),
    ("K.window_attend(q[:1], k, k, [1], [0], [300], 300, 2, out=out[:1])", False)])
def test_the_first_call_of_a_process_inside_a_capture(call, f32):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, call=call, f32=f32)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_at_once():
    """Each thread its own stream, workspaces and outputs (the calls share the device's error word and nothing else)."""
    q, k, v, ks = Wn.inputs([200, 1], [900, 5000], 8, 2, 128, BF, gap=0)
    pos, tab = torch.arange(q.shape[0], device="cuda"), K.rope_table(128)
    args = (q, k, v, [200, 1], ks, [900, 5000], 2048, 4)
    want, turned = K.window_attend(*args), K.qk_norm_rope(q, None, pos, tab)[0]
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [(K.window_attend(*args), K.qk_norm_rope(q, None, pos, tab)[0]) for _ in range(20)]
            s.synchronize()
            bad.extend(1 for a, b in got if not (torch.equal(a, want) and torch.equal(b, turned)))
            s.synchronize()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and K.window_check() == (K.OK, 0)


@pytest.mark.parametrize("ql,kl,window,dtype", [([1] * 5, [1, 90, 700, 4000, 9000], 8000, BF), ([1], [9000], 8000, F32),
                                                ([500, 30, 700], [500, 3000, 5000], 2048, BF), ([300], [3000], 2048, F32)])
def test_the_same_bits_every_time(ql, kl, window, dtype):
    q, k, v, ks = Wn.inputs(ql, kl, 4, 2, 128, dtype, gap=0)
    lse = [torch.empty(q.shape[:2], device="cuda") for _ in range(2)]
    want = K.window_attend(q, k, v, ql, ks, kl, window, 4, lse=lse[0])
    for _ in range(20):
        assert torch.equal(K.window_attend(q, k, v, ql, ks, kl, window, 4, lse=lse[1]), want)
        assert torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padded_batches(dtype):
    """Rows behind each prompt's own (padding) hold NaN and infinities: segments name the rows that count."""
    lens, pad = [70, 128, 3], 140
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.full((3 * pad, 2, 64), x, device="cuda", dtype=dtype) for x in (math.nan, math.inf))
    for b, n in enumerate(lens):
        for x in (k, v):
            x[b * pad:b * pad + n] = torch.randn((n, 2, 64), device="cuda", generator=g).to(dtype)
    q = torch.randn((sum(lens), 4, 64), device="cuda", generator=g).to(dtype)
    lse = torch.empty(q.shape[:2], device="cuda")
    starts = [b * pad for b in range(3)]
    out = K.window_attend(q, k, v, lens, starts, lens, 50, 2, lse=lse)
    Wn.check(out, lse, Wn.formula(q, k, v, lens, starts, lens, 50, 2, 0.125), q, k, 0.125, dtype, 128)
