"""The operators around the two-pool cache as cases to time: head norms with
the position rotation, window attention over a prompt, and decode attention of
a batch that shares a prefix.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the package's entry points; ``exact``
computes the same outputs in 64 bits from the operator's definition.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
M_PRIME = 128  # tokens per block


def listed():
    return [
        # one decode step of a batch of 32: one new token each, 16 heads x 128
        dict(name="rope_step", op="rope", tokens=32, hq=16, hk=16, d=128, rot=128, dtype="bf16", inter=False, far=8192),
        # one chunk of a chunked prefill: 4 requests x 2048 tokens
        dict(name="rope_chunk", op="rope", tokens=8192, hq=16, hk=16, d=128, rot=64, dtype="bf16", inter=True, far=32768),
        # a long prompt's tail at positions up to a million, shared key heads, an odd count
        dict(name="rope_long", op="rope", tokens=65537, hq=16, hk=4, d=128, rot=128, dtype="bf16", inter=False, far=1 << 20),
        # fp32 heads of 64, as the smallest configuration has them
        dict(name="rope_f32", op="rope", tokens=4099, hq=4, hk=4, d=64, rot=64, dtype="f32", inter=False, far=4096),
        # single tokens of a decode batch: 32 requests of up to 8192 tokens, window 128
        dict(name="win_step", op="win", batch=32, q_len=1, k_max=8192, hq=16, hk=16, d=128, window=128, sink=4, dtype="bf16"),
        # single tokens of a serving batch with the wide window, shared key heads
        dict(name="win_serve", op="win", batch=64, q_len=1, k_max=16384, hq=16, hk=4, d=128, window=4096, sink=0, dtype="bf16"),
        # one chunk of a chunked prefill at the end of 32768-token prompts, window 128
        dict(name="win_chunk", op="win", batch=4, q_len=2048, k_max=32768, hq=16, hk=16, d=128, window=128, sink=4, dtype="bf16"),
        # a whole 32768-token prompt under the wide window
        dict(name="win_prompt", op="win", batch=1, q_len=32768, k_max=32768, hq=16, hk=16, d=128, window=4096, sink=4, dtype="bf16"),
        # fp32, ragged prompts of odd lengths, heads of 64
        dict(name="win_f32", op="win", batch=3, q_len=1021, k_max=1021, hq=4, hk=4, d=64, window=256, sink=1, dtype="f32"),
        # decode of 4 requests behind a 16384-token prefix (the chunked prefill's shared half)
        dict(name="shared_small", op="shared", batch=4, prefix=16384, own=300, heads=16, d=128, dtype="bf16"),
        # decode of 32 requests behind a 131072-token prefix
        dict(name="shared_batch", op="shared", batch=32, prefix=131072, own=8192, heads=16, d=128, dtype="bf16"),
        # decode of 64 requests behind a million-token prefix
        dict(name="shared_long", op="shared", batch=64, prefix=1 << 20, own=4096, heads=16, d=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "win", "win", "shared"])
    if op == "rope":
        d = rng.choice([64, 128])
        return dict(op=op, tokens=_log_int(rng, 1, 65537), hq=rng.choice([4, 8, 16]), hk=rng.choice([1, 4, 16]), d=d,
                    rot=rng.choice([d, d // 2]), dtype=rng.choice(["bf16", "bf16", "f32"]), inter=rng.random() < 0.5,
                    far=_log_int(rng, 16, 1 << 20))
    if op == "win":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        hk = rng.choice([2, 4, 16])
        hq = hk * rng.choice([1, 2, 4])
        d = rng.choice([64, 128])
        window, sink = _log_int(rng, 16, 4096), rng.choice([0, 1, 4, 130])
        if rng.random() < 0.5:
            return dict(op=op, batch=_log_int(rng, 1, 64), q_len=1, k_max=_log_int(rng, 1, 16384), hq=hq, hk=hk, d=d,
                        window=window, sink=sink, dtype=dtype)
        batch = rng.choice([1, 2, 4])
        q_len = _log_int(rng, 2, (2048 if dtype == "f32" else 8192) // batch)
        return dict(op=op, batch=batch, q_len=q_len, k_max=_log_int(rng, q_len, 32768 // batch), hq=min(hq, 16), hk=min(hk, 4),
                    d=d, window=window, sink=sink, dtype=dtype)
    heads, d, dtype = rng.choice([(16, 128, "bf16"), (8, 128, "bf16"), (16, 64, "bf16"), (4, 64, "f32")])
    return dict(op=op, batch=_log_int(rng, 2, 64), prefix=M_PRIME * _log_int(rng, 1, 2048), own=_log_int(rng, 1, 4096),
                heads=heads, d=d, dtype=dtype)


# ---- inputs -----------------------------------------------------------------


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _normal(shape, dtype, g):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=g).to(dtype)


def _inv_freq(rot):
    return 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)


def _prepare_rope(c, seed):
    g, dt = _gen(seed, 1), DT[c["dtype"]]
    # a fused projection's output: query heads, key heads and value heads of a token in one row
    rows = _normal((c["tokens"], c["hq"] + 2 * c["hk"], c["d"]), dt, g)
    s = {"q": rows[:, :c["hq"]], "k": rows[:, c["hq"]:c["hq"] + c["hk"]],
         "pos": torch.randint(0, c["far"], (c["tokens"],), device="cuda", dtype=torch.int64, generator=g),
         "qw": 1 + 0.1 * _normal((c["d"],), torch.float32, g), "kw": 1 + 0.1 * _normal((c["d"],), torch.float32, g),
         "freq": torch.from_numpy(_inv_freq(c["rot"])).cuda()}
    if own:
        from heterogeneous_compressed_kv_gb300 import kvpool as K
        s["table"] = K.rope_table(c["rot"], inv_freq=_inv_freq(c["rot"]))
    return s


def _queries(c):
    """Queries of each request: one each, or ragged prompts of q_len down to half of it."""
    b = np.arange(c["batch"], dtype=np.int64)
    return c["q_len"] - b * (c["q_len"] // 2) // c["batch"]


def _lengths(c, seed):
    """Cached tokens of each request: up to k_max, at least its queries' own tokens; prompts are whole where k_max is q_len."""
    r = np.random.RandomState((int(seed) * 7919 + 3) & 0x7FFFFFFF)
    lo = min(c["q_len"], c["k_max"])
    return r.randint(lo, c["k_max"] + 1, c["batch"]).astype(np.int64)


def _prepare_win(c, seed):
    g, dt = _gen(seed, 2), DT[c["dtype"]]
    k_len = _lengths(c, seed)
    q_len = _queries(c)
    k_start = np.concatenate([[0], np.cumsum(k_len)[:-1]]).astype(np.int64)
    rows = int(k_len.sum())
    return {"q": _normal((int(q_len.sum()), c["hq"], c["d"]), dt, g), "k": _normal((rows, c["hk"], c["d"]), dt, g),
            "v": _normal((rows, c["hk"], c["d"]), dt, g), "q_len": q_len, "k_start": k_start, "k_len": k_len}


def _chain(alpha, x):
    """Entries of whole blocks: the fp32 fused multiply-add chain over a block's tokens (64-bit products and sums, each
    step rounded to 32 bits). alpha [H][128], x [blocks][128][H][D]."""
    acc = torch.zeros_like(x[:, 0], dtype=torch.float32)
    for i in range(M_PRIME):
        acc = (alpha[:, i].double()[None, :, None] * x[:, i].double() + acc.double()).float()
    return acc.to(x.dtype)


def _prepare_shared(c, seed):
    """A pool of one HCA layer whose requests share a prefix and then hold tokens of their own; the plain form keeps the
    same entries and windows as tensors."""
    g, dt, H, D, B = _gen(seed, 5), DT[c["dtype"]], c["heads"], c["d"], c["batch"]
    r = np.random.RandomState((int(seed) * 7919 + 6) & 0x7FFFFFFF)
    n_own = r.randint(1, c["own"] + 1, B).astype(np.int64)
    P, blocks = c["prefix"], c["prefix"] // M_PRIME
    gate = np.random.RandomState((int(seed) * 7919 + 7) & 0x7FFFFFFF).randn(1, H, M_PRIME).astype(np.float32)
    alpha = torch.softmax(torch.from_numpy(gate[0]).double(), -1).float().cuda()
    pool = req = None
    if own:
        from heterogeneous_compressed_kv_gb300 import kvpool as K
        total = blocks + int((n_own // M_PRIME).sum()) + B
        kd = K.F32 if dt == torch.float32 else K.BF16
        cfg = K.PoolConfig(m=4, m_prime=M_PRIME, n_win=M_PRIME, heads=H, head_dim=D, idx_heads=1, idx_dim=32, in_dtype=kd,
                           cache_dtype=kd, layer_kinds=[K.HCA], max_requests=B, max_blocks=total,
                           max_blocks_per_request=blocks + c["own"] // M_PRIME + 1, max_batch=B, max_top_k=0,
                           gate_csa=np.zeros((1, H, 4), np.float32), gate_hca=gate, gate_idx=np.zeros((1, 1, 4), np.float32))
        arena = torch.empty(K.required_bytes(cfg), dtype=torch.uint8, device="cuda")
        pool = K.Pool(cfg, arena)
        req = [pool.alloc_request() for _ in range(B)]
    hk, hv, win = [], [], None
    step = 1024 * M_PRIME
    for t0 in range(0, P, step):  # the prefix, once
        n = min(step, P - t0)
        k, v = _normal((n, H, D), dt, g), _normal((n, H, D), dt, g)
        if own:
            for u in range(0, n, 2048):
                pool.append([req[0]], [min(2048, n - u)], k[u:u + 2048], v[u:u + 2048], None)
        else:
            hk.append(_chain(alpha, k.view(-1, M_PRIME, H, D)))
            hv.append(_chain(alpha, v.view(-1, M_PRIME, H, D)))
        win = (k[-M_PRIME:].clone(), v[-M_PRIME:].clone())
    s = {"q": _normal((B, H, D), dt, g), "own": n_own}
    if own:
        for b in range(1, B):
            pool.share_prefix(req[b], req[0], P, win[0], win[1])
    most = int(max(n_own // M_PRIME))
    ek, ev = (torch.zeros((B, most, H, D), dtype=dt, device="cuda") for _ in range(2))
    wk, wv = (torch.zeros((B, M_PRIME, H, D), dtype=dt, device="cuda") for _ in range(2))
    for b in range(B):  # each request's own tokens
        n = int(n_own[b])
        k, v = _normal((n, H, D), dt, g), _normal((n, H, D), dt, g)
        if own:
            for u in range(0, n, 2048):
                pool.append([req[b]], [min(2048, n - u)], k[u:u + 2048], v[u:u + 2048], None)
            continue
        e = n // M_PRIME
        if e:
            ek[b, :e] = _chain(alpha, k[:e * M_PRIME].view(e, M_PRIME, H, D))
            ev[b, :e] = _chain(alpha, v[:e * M_PRIME].view(e, M_PRIME, H, D))
        wk[b], wv[b] = torch.cat([win[0], k])[-M_PRIME:], torch.cat([win[1], v])[-M_PRIME:]
    if own:
        s.update(pool=pool, req=np.array(req, np.int32), prefix=P, out=torch.empty((B, H, D), dtype=torch.float32, device="cuda"))
    else:
        s.update(hk=torch.cat(hk), hv=torch.cat(hv), ek=ek, ev=ev, wk=wk, wv=wv,
                 n_ent=torch.from_numpy(n_own // M_PRIME).cuda())
    return s


def prepare(case, seed):
    s = {"rope": _prepare_rope, "win": _prepare_win, "shared": _prepare_shared}[case["op"]](case, seed)
    s["case"] = case
    return s


# ---- plain forms ------------------------------------------------------------


def _rope_plain(x, w, ang, c):
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    rot, half = c["rot"], c["rot"] // 2
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :half], y[..., half:rot])
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([p, q], -1).flatten(-2) if c["inter"] else torch.cat([p, q], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _softmax_av(s, v):
    """softmax over the last axis (an empty row gives zeros) times v, and the log-sum-exp."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l), (m + torch.log(l)).squeeze(-1)


def _win_rows(q, k, v, pos, t, c):
    """Queries q [n][hq][d] at positions pos over keys k, v [m][hk][d] at positions t."""
    group = c["hq"] // c["hk"]
    qf = q.float().transpose(0, 1)  # [hq][n][d]
    kf, vf = (x.float().transpose(0, 1).repeat_interleave(group, 0) for x in (k, v))
    s = torch.matmul(qf, kf.transpose(1, 2)) / math.sqrt(c["d"])
    see = (t[None] <= pos[:, None]) & ((t[None] > pos[:, None] - c["window"]) | (t[None] < c["sink"]))
    o, l = _softmax_av(torch.where(see, s, torch.full_like(s, -math.inf)), vf)
    return o.transpose(0, 1).to(q.dtype), l.transpose(0, 1)


def _win_plain(s, c):
    q, k, v, W, S = s["q"], s["k"], s["v"], c["window"], c["sink"]
    if c["q_len"] == 1:  # single tokens: every request's visible keys, gathered into one padded batch
        k_len = torch.from_numpy(s["k_len"]).to(q.device, non_blocking=True)
        k_start = torch.from_numpy(s["k_start"]).to(q.device, non_blocking=True)
        w, n_s = min(W, int(s["k_len"].max())), min(S, int(s["k_len"].max()))
        lo = torch.clamp(k_len - w, min=0)
        t = torch.cat([torch.arange(n_s, device=q.device).expand(c["batch"], n_s),
                       lo[:, None] + torch.arange(w, device=q.device)], 1)
        see = t < k_len[:, None]
        see[:, :n_s] &= t[:, :n_s] < lo[:, None]
        rows = k_start[:, None] + torch.minimum(t, k_len[:, None] - 1)
        kf, vf = k[rows].float().transpose(1, 2), v[rows].float().transpose(1, 2)  # [b][hk][n][d]
        qf = q.float().view(c["batch"], c["hk"], c["hq"] // c["hk"], c["d"])
        sc = torch.matmul(qf, kf.transpose(2, 3)) / math.sqrt(c["d"])
        o, l = _softmax_av(torch.where(see[:, None, None], sc, torch.full_like(sc, -math.inf)), vf)
        return {"out": o.reshape(q.shape).to(q.dtype), "lse": l.reshape(c["batch"], c["hq"])}
    out, lse, at = [], [], 0
    for n, k0, kl in zip(s["q_len"].tolist(), s["k_start"].tolist(), s["k_len"].tolist()):
        for j in range(0, n, 1024):  # blocks of queries, each over the keys that it can see
            m = min(1024, n - j)
            p0 = kl - n + j
            lo, hi = max(0, p0 - W + 1), p0 + m
            t = torch.arange(lo, hi, device=q.device)
            if S and lo:
                t = torch.cat([torch.arange(min(S, lo), device=q.device), t])
            pos = torch.arange(p0, p0 + m, device=q.device)
            o, l = _win_rows(q[at + j:at + j + m], k[k0 + t], v[k0 + t], pos, t, c)
            out.append(o)
            lse.append(l)
        at += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _shared_scores(q, k, d):
    return torch.einsum("bhd,nhd->bhn", q, k.float()) / math.sqrt(d)


def _shared_plain(s, c):
    q = s["q"].float()
    ent = torch.arange(s["ek"].shape[1], device=q.device)[None] < s["n_ent"][:, None]  # [b][n]
    sh = _shared_scores(q, s["hk"], c["d"])
    se = torch.einsum("bhd,bnhd->bhn", q, s["ek"].float()) / math.sqrt(c["d"])
    se = torch.where(ent[:, None], se, torch.full_like(se, -math.inf))
    sw = torch.einsum("bhd,bnhd->bhn", q, s["wk"].float()) / math.sqrt(c["d"])
    m = torch.cat([sh, se, sw], -1).amax(-1, keepdim=True)
    sh, se, sw = torch.exp(sh - m), torch.exp(se - m), torch.exp(sw - m)
    l = sh.sum(-1) + se.sum(-1) + sw.sum(-1)
    o = torch.einsum("bhn,nhd->bhd", sh, s["hv"].float()) + torch.einsum("bhn,bnhd->bhd", se, s["ev"].float())
    return (o + torch.einsum("bhn,bnhd->bhd", sw, s["wv"].float())) / l[..., None]


def run(state):
    c = state["case"]
    if own:
        from heterogeneous_compressed_kv_gb300 import kvpool as K
        if c["op"] == "rope":
            q, k = K.qk_norm_rope(state["q"], state["k"], state["pos"], state["table"], state["qw"], state["kw"], eps=EPS,
                                  interleaved=c["inter"])
            return {"q": q, "k": k}
        if c["op"] == "win":
            lse = torch.empty(state["q"].shape[:2], dtype=torch.float32, device="cuda")
            out = K.window_attend(state["q"], state["k"], state["v"], state["q_len"], state["k_start"], state["k_len"],
                                  window=c["window"], n_sink=c["sink"], lse=lse)
            return {"out": out, "lse": lse}
        state["pool"].decode_attend_shared(0, state["req"], state["prefix"], state["q"], None, 0, state["out"])
        return {"out": state["out"]}
    if c["op"] == "rope":
        ang = state["pos"].double()[:, None] * state["freq"]
        return {"q": _rope_plain(state["q"], state["qw"], ang, c), "k": _rope_plain(state["k"], state["kw"], ang, c)}
    if c["op"] == "win":
        return _win_plain(state, c)
    return {"out": _shared_plain(state, c)}


# ---- the work of a pass -------------------------------------------------------


def work(case):
    c = case
    isz = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * n * isz + 8 * c["tokens"], "flops": 8 * n}
    if c["op"] == "win":
        # lengths are drawn from the seed; their means stand for them
        whole = c["k_max"] == c["q_len"]
        k_len = (c["q_len"] + c["k_max"]) / 2 if not whole else c["k_max"]
        q_len = float(_queries(c).mean())
        p = np.linspace(k_len - q_len, k_len - 1, min(int(q_len) + 1, 4096))
        win = np.minimum(p + 1, c["window"])
        pairs = float(np.mean(win + np.minimum(c["sink"], p + 1 - win))) * q_len * c["batch"]
        seen = min(k_len, q_len - 1 + c["window"] + c["sink"]) * c["batch"]
        rows = q_len * c["batch"] * c["hq"]
        return {"bytes": 2 * rows * c["d"] * isz + 4 * rows + 2 * seen * c["hk"] * c["d"] * isz,
                "flops": 4 * pairs * c["hq"] * c["d"]}
    row = c["heads"] * c["d"]
    own_rows = c["batch"] * (M_PRIME + c["own"] / 2 / M_PRIME)
    shared = c["prefix"] // M_PRIME
    return {"bytes": 2 * (shared + own_rows) * row * isz + c["batch"] * row * (isz + 4),
            "flops": 4 * row * (shared * c["batch"] + own_rows)}


# ---- 64 bits --------------------------------------------------------------------


def _exact_rope(s, c):
    res = {}
    theta = torch.outer(s["pos"].double(), s["freq"])
    turn = torch.complex(torch.cos(theta), torch.sin(theta))[:, None]
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        y = x / (x.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.double()
        rot = c["rot"]
        even, odd = ([2 * i for i in range(rot // 2)], [2 * i + 1 for i in range(rot // 2)]) if c["inter"] else (
            list(range(rot // 2)), list(range(rot // 2, rot)))
        z = torch.complex(y[..., even], y[..., odd]) * turn
        y[..., even], y[..., odd] = z.real, z.imag
        res[name] = y
    return res


def _exact_win(s, c):
    n_rows = s["q"].shape[0]
    out = torch.zeros((n_rows, c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((n_rows, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group, at = c["hq"] // c["hk"], 0
    for b in range(c["batch"]):
        n, k0, kl = int(s["q_len"][b]), int(s["k_start"][b]), int(s["k_len"][b])
        for j in range(0, n, 512):
            p = torch.arange(kl - n + j, kl - n + min(j + 512, n), device="cuda")
            first = max(0, int(p[0]) - c["window"] + 1)
            t = [i for i in range(min(c["sink"], first))] + [i for i in range(first, int(p[-1]) + 1)]
            t = torch.tensor(t, device="cuda")
            hidden = (t[None] > p[:, None]) | ((t[None] <= p[:, None] - c["window"]) & (t[None] >= c["sink"]))
            for h in range(c["hk"]):
                k, v = s["k"][k0 + t, h].double(), s["v"][k0 + t, h].double()
                for g in range(group):
                    a = s["q"][at + j:at + j + len(p), h * group + g].double() @ k.T / math.sqrt(c["d"])
                    a[hidden] = -math.inf
                    z = torch.logsumexp(a, -1)
                    out[at + j:at + j + len(p), h * group + g] = torch.exp(a - z[:, None]) @ v
                    lse[at + j:at + j + len(p), h * group + g] = z
        at += n
    return {"out": out, "lse": lse}


def _exact_shared(s, c):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        e = int(s["n_ent"][b])
        for h in range(c["heads"]):
            k = torch.cat([s["hk"][:, h], s["ek"][b, :e, h], s["wk"][b, :, h]]).double()
            v = torch.cat([s["hv"][:, h], s["ev"][b, :e, h], s["wv"][b, :, h]]).double()
            out[b, h] = torch.softmax(k @ s["q"][b, h].double() / math.sqrt(c["d"]), 0) @ v
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "win": _exact_win, "shared": _exact_shared}[case["op"]](s, case)
