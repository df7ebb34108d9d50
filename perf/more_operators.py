"""A paged cache held in 4 bits and what reads and shrinks it, and the rotation
by positions of several axes, as cases to time: tokens stored into the cache
(and read back as the values it stands for), attention over it with the weight
that each token got, eviction of the tokens that got least, and head norms with
a rotation by time, height and width.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the package's entry points; ``exact``
computes the same outputs in 64 bits from the operator's definition.

The cache's format: 16 neighbouring values of a head share an 8-bit scale s =
e4m3(amax / 6), amax their largest magnitude; each value is the nearest of 0,
0.5, 1, 1.5, 2, 3, 4, 6 times s, ties to the even code, with its sign. k_scale and
v_scale are powers of two that the whole cache's values are divided by first.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16
K_SCALE, V_SCALE = 1.0, 0.25


def listed():
    return [
        # one decode step of 64 requests with images in their prompts: time, height and width of each new token
        dict(name="axes_step", op="axes", tokens=64, hq=16, hk=16, d=128, rot=128, split="16,24,24", dtype="bf16", inter=False,
             far=8192),
        # a long prompt's tokens of video frames, shared key heads, an odd count
        dict(name="axes_video", op="axes", tokens=32769, hq=16, hk=4, d=128, rot=128, split="16,24,24", dtype="bf16", inter=False,
             far=32768),
        # the new tokens of a decode batch of 32 into the cache
        dict(name="store_step", op="store", batch=32, n_new=1, start=8192, hk=16, d=128, page=64, dtype="bf16"),
        # one chunk of a chunked prefill: 4 requests of up to 2048 tokens behind up to 32768
        dict(name="store_chunk", op="store", batch=4, n_new=2048, start=32768, hk=16, d=128, page=128, dtype="bf16"),
        # a decode batch: 32 requests of up to 8192 tokens
        dict(name="attend_step", op="attend", batch=32, q_len=1, k_max=8192, hq=16, hk=4, d=128, page=64, dtype="bf16", weigh=False),
        # a serving batch that keeps the tokens' weights for a later eviction
        dict(name="attend_weigh", op="attend", batch=64, q_len=1, k_max=16384, hq=16, hk=4, d=128, page=128, dtype="bf16", weigh=True),
        # one request behind a million tokens, every head with its own keys
        dict(name="attend_long", op="attend", batch=1, q_len=1, k_max=1 << 20, hq=16, hk=16, d=128, page=256, dtype="bf16", weigh=False),
        # fp32, small heads, a few drafted tokens each, odd lengths
        dict(name="attend_f32", op="attend", batch=5, q_len=3, k_max=3001, hq=4, hk=4, d=64, page=16, dtype="f32", weigh=True),
        # a chunk of a prompt behind a long cache
        dict(name="attend_chunk", op="attend", batch=2, q_len=1024, k_max=32768, hq=16, hk=4, d=128, page=128, dtype="bf16",
             weigh=False),
        # a few requests cut back to their heaviest 1024 tokens
        dict(name="evict_batch", op="evict", batch=16, k_max=4096, keep=1024, sink=4, recent=128, hk=4, d=128, page=64, dtype="bf16"),
        # long contexts cut back to 16384 tokens
        dict(name="evict_long", op="evict", batch=4, k_max=131072, keep=16384, sink=4, recent=1024, hk=8, d=128, page=128,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "store", "attend", "attend", "attend", "evict"])
    d, dtype, page = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice([16, 32, 64, 128, 256])
    if op == "axes":
        rot = rng.choice([d, d // 2])
        n, a = rot // 2, rng.randint(1, rot // 4)
        split = rng.choice([(n,), (a, n - a), (a, n // 2, n // 2 - a), (a, n // 2 - a, n // 4, n // 4)])
        return dict(op=op, tokens=_log_int(rng, 1, 32769), hq=rng.choice([4, 8, 16]), hk=rng.choice([1, 4, 16]), d=d, rot=rot,
                    split=",".join(str(x) for x in split), dtype=dtype, inter=rng.random() < 0.5, far=_log_int(rng, 16, 1 << 20))
    if op == "store":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, n_new=_log_int(rng, 1, 8192 // batch), start=_log_int(rng, 1, 32768),
                    hk=rng.choice([1, 2, 4, 16]), d=d, page=page, dtype=dtype)
    if op == "evict":
        k_max = _log_int(rng, 16, 65536)
        keep = _log_int(rng, 8, k_max)
        sink = rng.choice([0, 1, 4])
        return dict(op=op, batch=_log_int(rng, 1, min(64, max(1, 262144 // k_max))), k_max=k_max, keep=keep, sink=sink,
                    recent=rng.randint(0, (keep - sink) // 2), hk=rng.choice([1, 2, 4, 8]), d=d, page=page, dtype=dtype)
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 4, 8, 16] if hk <= 2 else [1, 2, 4])
    kind = rng.random()
    if kind < 0.7:  # one token to each request, or a few
        q_len = 1 if kind < 0.45 else rng.randint(2, 4)
        k_max = _log_int(rng, q_len, 262144)
        return dict(op=op, batch=_log_int(rng, 1, min(64, max(1, 524288 // k_max))), q_len=q_len, k_max=k_max, hq=hq, hk=hk, d=d,
                    page=page, dtype=dtype, weigh=rng.random() < 0.5)
    batch = rng.choice([1, 2])
    q_len = _log_int(rng, 65, (256 if dtype == "f32" else 1024) // batch)
    return dict(op=op, batch=batch, q_len=q_len, k_max=_log_int(rng, q_len, 16384 // batch), hq=min(hq, 16), hk=min(hk, 4), d=d,
                page=page, dtype=dtype, weigh=False)


# ---- inputs -----------------------------------------------------------------


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _host(seed, salt):
    return np.random.RandomState((int(seed) * 7919 + salt) & 0x7FFFFFFF)


def _normal(shape, dtype, g):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=g).to(dtype)


def _keys_values(n, c, g):
    """Tokens as a model makes them: key channels of unlike sizes, values of a smaller one."""
    size = torch.exp(0.5 * torch.randn((c["hk"], c["d"]), device="cuda", generator=g))
    k = (torch.randn((n, c["hk"], c["d"]), device="cuda", generator=g) * size).to(DT[c["dtype"]])
    return k, (0.3 * torch.randn((n, c["hk"], c["d"]), device="cuda", generator=g)).to(DT[c["dtype"]])


def _tables(pages, seed, salt, extra=0):
    """Rows of page ids in no order, `pages[i]` of them in row i, of `extra` pages more than all rows hold."""
    total = int(sum(pages)) + extra
    ids = _host(seed, salt).permutation(total).astype(np.int32)
    table, at = np.zeros((len(pages), max(int(max(pages)), 1)), np.int32), 0
    for i, n in enumerate(pages):
        table[i, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), total


def _quantize(x, scale):
    """Codes and scales of x [..., d] in the cache's format: packed codes [..., d / 2] and e4m3 scales [..., d / 16]."""
    f = (x.float() / scale).unflatten(-1, (-1, GROUP))
    amax = f.abs().amax(-1)
    s = torch.clamp(amax / torch.full_like(amax, 6.0), max=448.0).to(torch.float8_e4m3fn)
    w, a = s.float()[..., None], f.abs()
    code = ((a > 0.25 * w).int() + (a >= 0.75 * w) + (a > 1.25 * w) + (a >= 1.75 * w) + (a > 2.5 * w) + (a >= 3.5 * w) + (a > 5 * w))
    code = torch.where(w == 0, 0, code + 8 * (f < 0).int()).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), s


def _values(codes, s, scale):
    """The values, in 32 bits, that packed codes and scales stand for."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device) * scale
    x = torch.stack([level[(codes & 15).int()], level[(codes >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, GROUP)) * s.float()[..., None]).flatten(-2)


class _PlainCache:
    """The cache as tensors: packed codes and scales of keys and values by page and place in it."""

    def __init__(self, n_pages, c):
        self.page = c["page"]
        shape = (n_pages, c["page"], c["hk"])
        self.codes = [torch.zeros(shape + (c["d"] // 2,), dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(shape + (c["d"] // GROUP,), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]

    def place(self, table, seg, pos):
        """Page and place in it of the tokens at positions pos of table rows seg."""
        return table[seg, pos // self.page].long(), pos % self.page

    def store(self, k, v, at):
        for i, (x, scale) in enumerate(((k, K_SCALE), (v, V_SCALE))):
            codes, s = _quantize(x, scale)
            self.codes[i][at] = codes
            self.scales[i].view(torch.uint8)[at] = s.view(torch.uint8)

    def raw(self, which, at):
        return self.codes[which][at], self.scales[which].view(torch.uint8)[at].view(torch.float8_e4m3fn)

    def load(self, which, at):
        return _values(*self.raw(which, at), V_SCALE if which else K_SCALE)


def _ragged(starts, lens):
    """Segment and position of every token of a ragged batch."""
    seg = np.repeat(np.arange(len(lens)), lens)
    pos = np.arange(int(np.sum(lens))) - np.repeat(np.cumsum(lens) - lens, lens) + np.repeat(starts, lens)
    return torch.from_numpy(seg).cuda(), torch.from_numpy(pos).cuda()


def _own_cache(n_pages, c):
    from heterogeneous_compressed_kv_gb300 import kvpool as K
    pages = torch.zeros((n_pages, K.kv4_page_bytes(c["hk"], c["d"], c["page"])), dtype=torch.uint8, device="cuda")
    return K.Kv4Cache(pages, c["hk"], c["d"], c["page"], K_SCALE, V_SCALE)


def _fill(cache, table, lens, c, g, mine):
    for i, n in enumerate(lens.tolist()):
        for t0 in range(0, n, 1 << 16):
            k, v = _keys_values(min(1 << 16, n - t0), c, g)
            if mine:
                cache.store(k, v, table[i:i + 1], [t0], [k.shape[0]])
            else:
                pos = torch.arange(t0, t0 + k.shape[0], device="cuda")
                cache.store(k, v, cache.place(table, torch.full_like(pos, i), pos))


def _cut(lens, page):
    return (lens + page - 1) // page


def _split(c):
    """How many pairs turn by each axis."""
    return [int(x) for x in c["split"].split(",")]


def _prepare_axes(c, seed, mine):
    g, split = _gen(seed, 11), _split(c)
    # a fused projection's output: query heads, key heads and value heads of a token in one row
    rows = _normal((c["tokens"], c["hq"] + 2 * c["hk"], c["d"]), DT[c["dtype"]], g)
    inv = 10000.0 ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])
    axes = [a for a, n in enumerate(split) for _ in range(n)]
    s = {"q": rows[:, :c["hq"]], "k": rows[:, c["hq"]:c["hq"] + c["hk"]], "freq": torch.from_numpy(inv).cuda(),
         "pos": torch.randint(0, c["far"], (c["tokens"], len(split)), device="cuda", dtype=torch.int64, generator=g),
         "qw": 1 + 0.1 * _normal((c["d"],), torch.float32, g), "kw": 1 + 0.1 * _normal((c["d"],), torch.float32, g),
         "axes": axes, "axis_of": torch.tensor(axes, device="cuda")}
    if mine:
        from heterogeneous_compressed_kv_gb300 import kvpool as K
        s["table"] = K.rope_table(c["rot"], inv_freq=inv)
    return s


def _spread(lo, hi, n, seed, salt):
    return _host(seed, salt).randint(lo, hi + 1, n).astype(np.int64)


def _prepare_store(c, seed, mine):
    g = _gen(seed, 12)
    n_new = c["n_new"] - np.arange(c["batch"], dtype=np.int64) * (c["n_new"] // 2) // c["batch"]
    start = _spread(0, c["start"], c["batch"], seed, 13)
    table, total = _tables(_cut(start + n_new, c["page"]), seed, 14)
    k, v = _keys_values(int(n_new.sum()), c, g)
    cache = _own_cache(total, c) if mine else _PlainCache(total, c)
    return {"cache": cache, "table": table, "start": start, "n_new": n_new, "k": k, "v": v}


def _prepare_attend(c, seed, mine):
    g = _gen(seed, 15)
    lo = c["k_max"] if c["batch"] == 1 else min(c["q_len"], c["k_max"])
    k_len = _spread(lo, c["k_max"], c["batch"], seed, 16)
    q_len = c["q_len"] - np.arange(c["batch"], dtype=np.int64) * (c["q_len"] // 2) // c["batch"]
    table, total = _tables(_cut(k_len, c["page"]), seed, 17)
    q = _normal((int(q_len.sum()), c["hq"], c["d"]), DT[c["dtype"]], g)
    cache = _own_cache(total, c) if mine else _PlainCache(total, c)
    _fill(cache, table, k_len, c, g, mine)
    w = torch.zeros((c["batch"], c["hk"], c["k_max"]), device="cuda") if c["weigh"] else None
    return {"cache": cache, "table": table, "q": q, "q_len": q_len, "k_len": k_len, "weights": w}


def _prepare_evict(c, seed, mine):
    g = _gen(seed, 18)
    k_len = _spread(max(c["k_max"] // 2, c["keep"]), c["k_max"], c["batch"], seed, 19)
    n, need = _cut(k_len, c["page"]), _cut(np.minimum(k_len, c["keep"]), c["page"])
    both, total = _tables(np.concatenate([n, need]), seed, 20)
    table, out_table = both[:c["batch"]], both[c["batch"]:, :max(int(need.max()), 1)].contiguous()
    cache = _own_cache(total, c) if mine else _PlainCache(total, c)
    _fill(cache, table, k_len, c, g, mine)
    # most tokens got next to nothing, some nothing at all, and equal weights are about
    w = torch.exp(3 * torch.randn((c["batch"], c["hk"], int(k_len.max())), device="cuda", generator=g) - 8)
    w[..., ::7] = w[..., ::7].bfloat16().float()
    w[..., 3::11] = 0
    return {"cache": cache, "table": table, "out_table": out_table, "k_len": k_len, "weights": w}


PREPARE = {"axes": _prepare_axes, "store": _prepare_store, "attend": _prepare_attend, "evict": _prepare_evict}


def prepare(case, seed):
    if own:
        s = PREPARE[case["op"]](case, seed, True)
    else:
        s = PREPARE[case["op"]](case, seed, False)
    s["case"] = case
    return s


# ---- plain forms ------------------------------------------------------------


def _axes_plain(x, w, ang, c):
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    rot, half = c["rot"], c["rot"] // 2
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :half], y[..., half:rot])
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([p, q], -1).flatten(-2) if c["inter"] else torch.cat([p, q], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _back(s, c, at):
    """Keys and values read back."""
    return {name: s["cache"].load(i, at).to(DT[c["dtype"]]) for i, name in enumerate(("k", "v"))}


def _store_plain(s, c):
    at = s["cache"].place(s["table"], *_ragged(s["start"], s["n_new"]))
    s["cache"].store(s["k"], s["v"], at)
    return _back(s, c, at)


def _attend_plain(s, c):
    out, lse, at, w, G = [], [], 0, s["weights"], c["hq"] // c["hk"]
    for i, (n, kl) in enumerate(zip(s["q_len"].tolist(), s["k_len"].tolist())):
        pos = torch.arange(kl, device="cuda")
        place = s["cache"].place(s["table"], torch.full_like(pos, i), pos)
        k, v = (s["cache"].load(x, place).transpose(0, 1) for x in range(2))  # [hk][keys][d]
        q = s["q"][at:at + n].float().view(n, c["hk"], G, c["d"]).permute(1, 0, 2, 3).reshape(c["hk"], n * G, c["d"])
        sc = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(c["d"])
        if n > 1:
            hidden = pos[None] > torch.arange(kl - n, kl, device="cuda").repeat_interleave(G)[:, None]
            sc = sc.masked_fill(hidden, -math.inf)
        m = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - m)
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / l
        out.append(o.view(c["hk"], n, G, c["d"]).transpose(0, 1).reshape(n, c["hq"], c["d"]).to(s["q"].dtype))
        lse.append((m + torch.log(l)).view(c["hk"], n, G).transpose(0, 1).reshape(n, c["hq"]))
        if w is not None:
            w[i, :, :kl] = (p / l).sum(1)
        at += n
    res = {"out": torch.cat(out), "lse": torch.cat(lse)}
    if w is not None:
        res["weights"] = w
    return res


def _evict_plain(s, c):
    keep, sink, recent, w = c["keep"], c["sink"], c["recent"], s["weights"]
    index = torch.full((c["batch"], c["hk"], keep), -1, dtype=torch.int32, device="cuda")
    left = torch.zeros((c["batch"], c["hk"], keep), device="cuda")
    heads, cache = torch.arange(c["hk"], device="cuda"), s["cache"]
    for i, kl in enumerate(s["k_len"].tolist()):
        n = min(kl, keep)
        if kl <= keep:
            idx = torch.arange(kl, device="cuda").expand(c["hk"], kl)
        else:
            order = torch.sort(w[i, :, sink:kl - recent], dim=-1, descending=True, stable=True).indices
            best = torch.sort(order[:, :keep - sink - recent] + sink, dim=-1).values
            first, last = (torch.arange(a, b, device="cuda").expand(c["hk"], b - a) for a, b in ((0, sink), (kl - recent, kl)))
            idx = torch.cat([first, best, last], -1)
        index[i, :, :n] = idx.int()
        left[i, :, :n] = torch.gather(w[i], 1, idx)
        seg = torch.full((n,), i, device="cuda")
        page, slot = cache.place(s["table"], seg[:, None], idx.T)  # [n][hk]
        to = cache.place(s["out_table"], seg, torch.arange(n, device="cuda"))
        for x in (*cache.codes, *(y.view(torch.uint8) for y in cache.scales)):
            x[to] = x[page, slot, heads[None]]
    lens = np.minimum(s["k_len"], keep)
    return {"index": index, "weights": left, **_back(s, c, cache.place(s["out_table"], *_ragged(np.zeros_like(lens), lens)))}


def run(state):
    c = state["case"]
    if own:
        from heterogeneous_compressed_kv_gb300 import kvpool as K
        if c["op"] == "axes":
            q, k = K.qk_norm_rope(state["q"], state["k"], state["pos"], state["table"], state["qw"], state["kw"], eps=EPS,
                                  interleaved=c["inter"], axes=state["axes"])
            return {"q": q, "k": k}
        if c["op"] == "store":
            state["cache"].store(state["k"], state["v"], state["table"], state["start"], state["n_new"])
            k, v = state["cache"].load(state["table"], state["start"], state["n_new"], dtype=DT[c["dtype"]])
            return {"k": k, "v": v}
        if c["op"] == "attend":
            lse = torch.empty(state["q"].shape[:2], dtype=torch.float32, device="cuda")
            out = state["cache"].attend(state["q"], state["table"], state["q_len"], state["k_len"], lse=lse,
                                        weights=state["weights"], decay=0.0)
            res = {"out": out, "lse": lse}
            if state["weights"] is not None:
                res["weights"] = state["weights"]
            return res
        index, left = state["cache"].evict(state["table"], state["k_len"], state["weights"], c["keep"], state["out_table"],
                                           n_sink=c["sink"], n_recent=c["recent"])
        lens = np.minimum(state["k_len"], c["keep"])
        k, v = state["cache"].load(state["out_table"], np.zeros_like(lens), lens, dtype=DT[c["dtype"]])
        return {"index": index, "weights": left, "k": k, "v": v}
    if c["op"] == "axes":
        ang = state["pos"][:, state["axis_of"]].double() * state["freq"]
        return {"q": _axes_plain(state["q"], state["qw"], ang, c), "k": _axes_plain(state["k"], state["kw"], ang, c)}
    return {"store": _store_plain, "attend": _attend_plain, "evict": _evict_plain}[c["op"]](state, c)


# ---- the work of a pass -------------------------------------------------------


def work(case):
    c = case
    isz = 2 if c["dtype"] == "bf16" else 4
    row = c["hk"] * c["d"] * (0.5 + 1 / GROUP) * 2  # a token's keys and values in the cache
    if c["op"] == "axes":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * n * isz + 8 * c["tokens"] * len(_split(c)), "flops": 8 * n}
    if c["op"] == "store":  # tokens in, the cache written, the values it stands for out
        n = float((c["n_new"] - np.arange(c["batch"]) * (c["n_new"] // 2) // c["batch"]).sum())
        v = 2 * n * c["hk"] * c["d"]
        return {"bytes": 2 * v * isz + n * row, "flops": 12 * v}
    if c["op"] == "attend":  # lengths are drawn from the seed; their means stand for them
        k_len = c["k_max"] if c["batch"] == 1 else (c["k_max"] + min(c["q_len"], c["k_max"])) / 2
        q_len = float((c["q_len"] - np.arange(c["batch"]) * (c["q_len"] // 2) // c["batch"]).mean())
        pairs = c["batch"] * c["hq"] * q_len * (k_len - (q_len - 1) / 2)
        rows = c["batch"] * q_len * c["hq"]
        weights = 4 * c["batch"] * c["hk"] * k_len if c["weigh"] else 0
        return {"bytes": c["batch"] * k_len * row + rows * (2 * c["d"] * isz + 4) + weights, "flops": 4 * pairs * c["d"]}
    k_len = (c["k_max"] + max(c["k_max"] // 2, c["keep"])) / 2
    n = c["batch"] * min(k_len, c["keep"])
    return {"bytes": 4 * c["batch"] * c["hk"] * k_len + 2 * n * row + n * c["hk"] * (8 + 2 * c["d"] * isz),
            "flops": 2 * n * c["hk"] * c["d"] + c["batch"] * c["hk"] * k_len}


# ---- 64 bits --------------------------------------------------------------------


def _exact_axes(s, c):
    res = {}
    theta = torch.stack([s["pos"][:, a].double() * s["freq"][i] for i, a in enumerate(s["axes"])], -1)
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


def _grid8():
    """The finite values of e4m3, from 0 to 448, in order: value i has the even mantissa where i is even."""
    return [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(x, grid):
    """x >= 0 in 64 bits to the nearest value of grid (ascending), ties to the even place, beyond the last one to it."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    i = torch.searchsorted(g, x.contiguous()).clamp(1, len(grid) - 1)
    down, up = x - g[i - 1], g[i] - x
    return g[torch.where((down < up) | ((down == up) & (i % 2 == 1)), i - 1, i)]


def _rounded(x, scale):
    """What the cache holds of x [..., d], in 64 bits."""
    f = (x.double() / scale).unflatten(-1, (-1, GROUP))
    six = (f.abs().amax(-1, keepdim=True).float() / torch.full((1,), 6.0, device=x.device)).double()  # the quotient is fp32's
    s = _nearest(six, _grid8())
    code = _nearest(torch.where(s > 0, f.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(f)), LEVELS)
    return (torch.copysign(code, f) * s * scale).flatten(-2)


def _exact_store(s, c):
    return {"k": _rounded(s["k"], K_SCALE), "v": _rounded(s["v"], V_SCALE)}


def _exact_load(s, which, b, pos, head):
    codes, sc = s["cache"].raw(which, s["cache"].place(s["table"], torch.full_like(pos, b), pos))
    codes, sc = codes[:, head], sc[:, head]
    level = torch.tensor([x * (-1.0) ** (i // 8) for i, x in enumerate(LEVELS * 2)], dtype=torch.float64, device="cuda")
    x = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device="cuda")
    x[:, 0::2], x[:, 1::2] = level[(codes % 16).int()], level[(codes // 16).int()]
    scale = V_SCALE if which else K_SCALE
    return x * sc.double().repeat_interleave(GROUP, 1) * scale


def _exact_attend(s, c):
    rows, G = s["q"].shape[0], c["hq"] // c["hk"]
    out = torch.zeros((rows, c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, c["hq"]), dtype=torch.float64, device="cuda")
    w = torch.zeros((c["batch"], c["hk"], c["k_max"]), dtype=torch.float64, device="cuda")
    at = 0
    for b in range(c["batch"]):
        n, kl = int(s["q_len"][b]), int(s["k_len"][b])
        pos = torch.arange(kl, device="cuda")
        for h in range(c["hk"]):
            k, v = (_exact_load(s, i, b, pos, h) for i in range(2))
            for g in range(G):
                a = s["q"][at:at + n, h * G + g].double() @ k.T / math.sqrt(c["d"])
                a[pos[None] > torch.arange(kl - n, kl, device="cuda")[:, None]] = -math.inf
                z = torch.logsumexp(a, -1)
                p = torch.exp(a - z[:, None])
                out[at:at + n, h * G + g] = p @ v
                lse[at:at + n, h * G + g] = z
                w[b, h, :kl] += p.sum(0)
        at += n
    res = {"out": out, "lse": lse}
    if c["weigh"]:
        res["weights"] = w
    return res


def _exact_evict(s, c):
    keep, w = c["keep"], s["weights"].cpu().numpy()
    index = np.full((c["batch"], c["hk"], keep), -1, np.int32)
    left = np.zeros((c["batch"], c["hk"], keep), np.float64)
    ks, vs = [], []
    for b in range(c["batch"]):
        kl = int(s["k_len"][b])
        n = min(kl, keep)
        k, v = (torch.empty((n, c["hk"], c["d"]), dtype=torch.float64, device="cuda") for _ in range(2))
        for h in range(c["hk"]):
            rank = w[b, h, :kl].astype(np.float64)
            rank[:c["sink"]] = np.inf
            rank[kl - c["recent"]:] = np.inf
            idx = np.sort(np.lexsort((np.arange(kl), -rank))[:n])  # heaviest first, then the lowest place
            index[b, h, :n], left[b, h, :n] = idx, w[b, h, idx]
            pos = torch.from_numpy(idx).cuda()
            k[:, h], v[:, h] = (_exact_load(s, i, b, pos, h) for i in range(2))
        ks.append(k)
        vs.append(v)
    return {"index": torch.from_numpy(index), "weights": torch.from_numpy(left), "k": torch.cat(ks), "v": torch.cat(vs)}


def exact(case, seed):
    s = PREPARE[case["op"]](case, seed, False)
    return {"axes": _exact_axes, "store": _exact_store, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](s, case)
