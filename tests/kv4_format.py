"""The 4-bit cache's format and its attention in 64 bits, on the CPU and apart from the kernels."""
import math

import numpy as np
import torch

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def nearest(x, grid):
    """x >= 0 to the nearest value of grid, ties to the even place, beyond the last one to it (float64 arrays)."""
    g = np.array(grid)
    i = np.clip(np.searchsorted(g, x), 1, len(g) - 1)
    down, up = x - g[i - 1], g[i] - x
    return g[np.where((down < up) | ((down == up) & (i % 2 == 1)), i - 1, i)]


def held(x, scale=1.0):
    """What the cache holds of x [..., dim] (float32 or bfloat16), in float64."""
    f = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        f = (f / np.float32(scale)).reshape(*f.shape[:-1], -1, 16)
        amax = np.abs(f).max(-1, keepdims=True)
        bad = ~np.isfinite(f).all(-1, keepdims=True)
        s = nearest(np.where(bad, 0, amax / np.float32(6)).astype(np.float64), E4M3)
        f = f.astype(np.float64)
        code = nearest(np.where(s > 0, np.abs(np.where(bad, 0, f)) / np.where(s > 0, s, 1), 0), LEVELS)
        y = np.where(bad, np.nan, np.copysign(code, f) * s * scale)
    return torch.from_numpy(y.reshape(x.shape))


def attend(q, k, v, q_len, k_len, scale):
    """(out, lse, weights [hk][k_len], error scales) of one segment in float64: q [q_len][hq][d], k and v [k_len][hk][d]
    as held.  The error scales are a bound of sum |q k| scale for each row, sum p |v| and sum |v|."""
    n, hq, d = q.shape
    hk = k.shape[1]
    G = hq // hk
    q = q.double().cpu()
    out, lse, size, mag = torch.zeros(n, hq, d).double(), torch.full((n, hq), -math.inf).double(), torch.zeros(n, hq).double(), \
        torch.zeros(n, hq, d).double()
    flat = torch.zeros(n, hq, d).double()
    w = torch.zeros(hk, k_len).double()
    for h in range(hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = q[:, h] @ kh.T * scale
        hidden = torch.arange(k_len)[None] > torch.arange(k_len - n, k_len)[:, None]
        s = s.masked_fill(hidden, -math.inf)
        for j in range(n):
            if k_len == 0 or bool(hidden[j].all()):
                continue
            z = torch.logsumexp(s[j], 0)
            p = torch.exp(s[j] - z)
            p = torch.where(hidden[j], torch.zeros_like(p), p)
            seen = ~hidden[j]
            out[j, h], lse[j, h] = p[seen] @ vh[seen], z
            mag[j, h], flat[j, h] = p[seen] @ vh[seen].abs(), vh[seen].abs().sum(0)
            size[j, h] = (q[j, h].abs() @ kh[seen].abs().T * abs(scale)).max()
            w[h // G] += p
    return out, lse, w, size, mag, flat
