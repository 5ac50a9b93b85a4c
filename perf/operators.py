"""What the serving operators around the compressed cache cost, and their plain forms.

Four operators, each with its listed cases and a range that `draw` samples:

  rope    RMS norm of every query and key head with the position rotation in the same pass
          (one position per token, or several axes), from slices of a fused QKV projection;
  cross   attention of ragged query runs over the compressed cache of an encoder's states
          (no causal mask, another length on either side);
  fork    rows of the block table forked (full pages shared, the partly filled page copied in
          every layer), the children given slots for new tokens, then freed;
  evict   rows forked, compacted to a list of kept tokens (records gathered into fresh pages
          in every layer), then freed.

With `own` false, `run` computes them with elementary torch operations; with `own` true it
makes the calls of `kv_cache_vector_07_b200.tqkv`.  `exact` gives the computed numbers from
the definitions in 64 bits.  The pages hold bytes and tables of integers: those are compared
as they are.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

PAGE = 64


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step's tokens of a small batch: the launch is the cost
        {"name": "rope_decode", "op": "rope", "n": 4, "hq": 32, "hk": 8, "d": 128, "rot": 128, "style": "half",
         "axes": 1, "dtype": "bf16", "norm": True, "far": 262144},
        # a long prefill chunk, 32 query and 8 key heads of 128
        {"name": "rope_prefill", "op": "rope", "n": 32768, "hq": 32, "hk": 8, "d": 128, "rot": 128, "style": "half",
         "axes": 1, "dtype": "bf16", "norm": True, "far": 32768},
        # image and video tokens: three axes, an odd count of tokens
        {"name": "rope_axes", "op": "rope", "n": 8191, "hq": 32, "hk": 8, "d": 128, "rot": 128, "style": "half",
         "axes": 3, "dtype": "bf16", "norm": True, "far": 4096},
        # float32, neighbouring pairs, a part of each head rotated, no norm
        {"name": "rope_partial_f32", "op": "rope", "n": 1000, "hq": 12, "hk": 4, "d": 64, "rot": 48, "style": "pairs",
         "axes": 1, "dtype": "f32", "norm": False, "far": 100000},
        # one new token of every sequence against its encoder states
        {"name": "cross_decode", "op": "cross", "b": 32, "maxq": 1, "maxkv": 2048, "hq": 32, "hk": 8, "d": 128,
         "page": PAGE, "codec": "k3v4"},
        # short prompts against encoder states, ragged on both sides
        {"name": "cross_prompt", "op": "cross", "b": 8, "maxq": 77, "maxkv": 4096, "hq": 32, "hk": 8, "d": 128,
         "page": PAGE, "codec": "k5v4"},
        # long runs against long encoder states: the tensor cores are the cost
        {"name": "cross_long", "op": "cross", "b": 8, "maxq": 1024, "maxkv": 8192, "hq": 32, "hk": 8, "d": 128,
         "page": PAGE, "codec": "k3v4"},
        # FP8 keys, small pages, five heads a group, heads of 64, some runs and states empty
        {"name": "cross_odd", "op": "cross", "b": 7, "maxq": 333, "maxkv": 1501, "hq": 10, "hk": 2, "d": 64,
         "page": 16, "codec": "k8v4"},
        # a small beam step
        {"name": "fork_beam", "op": "fork", "layers": 2, "blocks": 256, "hk": 8, "d": 128, "page": PAGE,
         "codec": "k3v4", "parents": 2, "each": 2, "plen": 1000, "new": 1},
        # sampling many continuations of long prompts, every layer of a cache
        {"name": "fork_many", "op": "fork", "layers": 32, "blocks": 512, "hk": 8, "d": 128, "page": PAGE,
         "codec": "k3v4", "parents": 4, "each": 15, "plen": 4001, "new": 5},
        # rejected draft tokens and a window: few rows, short
        {"name": "evict_short", "op": "evict", "layers": 2, "blocks": 128, "hk": 8, "d": 128, "page": PAGE,
         "codec": "k5v4", "rows": 3, "len": 700, "keep": 0.7, "sink": 300},
        # half of every long row evicted, all layers
        {"name": "evict_long", "op": "evict", "layers": 8, "blocks": 2048, "hk": 8, "d": 128, "page": PAGE,
         "codec": "k3v4", "rows": 8, "len": 8190, "keep": 0.5, "sink": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cross", "fork", "evict"])
    if op == "rope":
        d = rng.choice([64, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.randint(1, 4)
        rot = rng.choice([d, d, d // 2, d // 4 * 3])
        return {"op": op, "n": _log(rng, 1, 32768 * 40 * 128 // ((hq + hk) * d)), "hq": hq, "hk": hk, "d": d,
                "rot": rot, "style": rng.choice(["half", "pairs"]), "axes": rng.choice([1, 1, 2, 3]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]) if hq <= 16 else "bf16", "norm": rng.random() < 0.75,
                "far": _log(rng, 64, 262144)}
    if op == "cross":
        d = rng.choice([64, 128, 128])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.randint(1, 8 if hk <= 4 else 4)
        b, kv = _log(rng, 1, 32), _log(rng, 1, 8192)
        top = min(1024, max(1, 8 * 32 * 1024 * 8192 // (2 * b * hq * kv)))
        return {"op": op, "b": b, "maxq": _log(rng, 1, top), "maxkv": kv, "hq": hq, "hk": hk, "d": d,
                "page": rng.choice([64, 64, 32, 16]), "codec": rng.choice(["k3v4", "k5v4", "k8v4"])}
    hk, layers = rng.choice([2, 4, 8]), _log(rng, 1, 16)
    c = {"op": op, "layers": layers, "hk": hk, "d": rng.choice([64, 128]), "page": rng.choice([64, 64, 32, 16]),
         "codec": rng.choice(["k3v4", "k5v4", "k8v4"])}
    if op == "fork":
        c |= {"parents": rng.randint(1, 4), "each": rng.randint(1, 8), "plen": _log(rng, 1, 4001), "new": rng.randint(1, 9)}
        per = -(-c["plen"] // c["page"])
        c["blocks"] = c["parents"] * (per + 2 * c["each"]) + rng.randint(0, 100)
    else:
        c |= {"rows": rng.randint(1, 6), "len": _log(rng, 1, 4001), "keep": round(rng.uniform(0.05, 1.0), 2),
              "sink": rng.choice([0, 4, 100])}
        c["blocks"] = c["rows"] * (2 * -(-c["len"] // c["page"]) + 2) + rng.randint(0, 100)
    return c


def _lens(case, what, n, most, some_empty):
    """Ragged lengths that belong to the case (not to the seed), the first the longest."""
    r = random.Random("%s %s %d %d" % (case["op"], what, n, most))
    got = [most] + [max(1, int(most * r.uniform(0.4, 1.0))) for _ in range(n - 1)]
    if some_empty and n >= 5:
        got[2], got[-1] = 0, min(1, most)
    return got


def _codec(case):
    return {"k3v4": (2, True, 4), "k5v4": (4, True, 4), "k8v4": (8, False, 4)}[case["codec"]]


def _fields(case):
    """[(name, byte offset in a page, bytes per token)], and the bytes of a page."""
    kb, qjl, vb = _codec(case)
    d, P = case["d"], case["page"]
    sizes = [("kc", d if kb == 8 else d * kb // 8)] + ([("ks", d // 8)] if qjl else []) + [("kn", 2)]
    sizes += ([("kr", 2)] if qjl else []) + [("vc", d * vb // 8), ("vn", 2)]
    got, off = [], 0
    for name, n in sizes:
        got.append((name, off, n))
        off += (P * n + 15) // 16 * 16
    return got, off


def _token_bytes(case):
    return sum(n for _, _, n in _fields(case)[0])


def _cross_lens(case):
    return (_lens(case, "q", case["b"], case["maxq"], case["maxq"] > 1), _lens(case, "kv", case["b"], case["maxkv"], True))


def _evict_lens(case):
    lens = _lens(case, "len", case["rows"], case["len"], False)
    kept = [max(1, int(n * case["keep"])) for n in lens]
    return lens, kept, [min(case["sink"], k) for k in kept]


def work(case):
    if case["op"] == "rope":
        es = 2 if case["dtype"] == "bf16" else 4
        vals = case["n"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * es * vals + 4 * case["n"] * case["axes"] + 2 * case["rot"] + 2 * case["d"] * es,
                "flops": 10 * vals}
    if case["op"] == "cross":
        ql, kl = _cross_lens(case)
        seen = sum(k for q, k in zip(ql, kl) if q)
        return {"bytes": seen * case["hk"] * _token_bytes(case) + 2 * 2 * sum(ql) * case["hq"] * case["d"],
                "flops": 4 * case["d"] * case["hq"] * sum(q * k for q, k in zip(ql, kl))}
    P, page = case["page"], _fields(case)[1] * case["hk"]
    if case["op"] == "fork":
        lens = _lens(case, "plen", case["parents"], case["plen"], False)
        copies = case["each"] * sum(n % P != 0 for n in lens)
        entries = case["each"] * sum(-(-n // P) for n in lens)
        return {"bytes": 2 * copies * page * case["layers"] + 4 * (case["blocks"] + 6 * entries), "flops": entries}
    lens, kept, sink = _evict_lens(case)
    copies = sum(n % P != 0 for n in lens)
    moved = sum(k - s // P * P for k, s in zip(kept, sink))
    return {"bytes": 2 * copies * page * case["layers"] + 2 * moved * case["hk"] * case["layers"] * _token_bytes(case)
            + 4 * (case["blocks"] + sum(kept) + 6 * sum(-(-n // P) for n in lens)), "flops": moved}


# ---------------------------------------------------------------------------------------
# the data-independent parameters of the codec, from their definitions
# ---------------------------------------------------------------------------------------
def _draws(seed, stream, count):
    i = np.arange(count, dtype=np.uint64) + np.uint64(stream << 32) + np.uint64(1)
    z = np.uint64(seed) + i * np.uint64(0x9E3779B97F4A7C15)
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


@functools.lru_cache(maxsize=None)
def _signs(d, seed):
    return torch.from_numpy(np.where(_draws(seed, 0, d) >> np.uint64(63), -1.0, 1.0))


@functools.lru_cache(maxsize=None)
def _projection(d, seed):
    u = _draws(seed, 1, d * d).reshape(-1, 2) >> np.uint64(11)
    rad = np.sqrt(-2.0 * np.log((u[:, 0].astype(np.float64) + 1.0) * 2.0 ** -53))
    ang = 2.0 * np.pi * u[:, 1].astype(np.float64) * 2.0 ** -53
    S = np.stack([rad * np.cos(ang), rad * np.sin(ang)], 1).reshape(d, d)
    return torch.from_numpy(S).to(torch.bfloat16).to(torch.float64)


@functools.lru_cache(maxsize=None)
def _magnitudes(d, bits):
    """Positive levels of the Lloyd-Max quantizer of one coordinate of a random unit vector."""
    h, a = 1 << (bits - 1), (d - 3) / 2
    x, w = np.polynomial.legendre.leggauss(200)
    pos = 2.5 / math.sqrt(d) * (np.arange(h) + 0.5) / h
    for _ in range(20000):
        edge = np.concatenate([[0.0], 0.5 * (pos[1:] + pos[:-1]), [min(1.0, 12 / math.sqrt(d))]])
        t = 0.5 * (edge[1:] + edge[:-1])[:, None] + 0.5 * (edge[1:] - edge[:-1])[:, None] * x
        f = w * np.exp(a * np.log1p(-t * t))
        new = (f * t).sum(1) / f.sum(1)
        if np.abs(new - pos).max() < 1e-15:
            break
        pos = new
    return torch.from_numpy(new.astype(np.float32)).to(torch.float64)


def _hadamard(d, device, dtype):
    i = torch.arange(d, device=device)
    par = i[:, None] & i[None, :]
    for s in (8, 4, 2, 1):
        par = par ^ (par >> s)
    return 1 - 2 * (par & 1).to(dtype)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rope_inputs(case, seed):
    g = _generator(seed)
    n, hq, hk, d, ax = case["n"], case["hq"], case["hk"], case["d"], case["axes"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = torch.randn((n, (hq + 2 * hk), d), generator=g, device="cuda")
    qkv[:, :, 5] *= 8.0                                      # a channel that stands out, as projections have
    qkv = qkv.to(dt)
    weight = [(1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]
    if ax == 1:
        pos = torch.randint(0, case["far"], (1, n), generator=g, device="cuda", dtype=torch.int32)
    else:
        pos = torch.randint(0, case["far"], (ax, n), generator=g, device="cuda", dtype=torch.int32)
        pos[1:] %= 256                                       # heights and widths are short, times are not
    pairs = case["rot"] // 2
    inv = (500000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).to(torch.float32).cuda()
    axis = [p * ax // pairs for p in range(pairs)]           # contiguous sections of pairs, one for each axis
    return {"qkv": qkv, "qw": weight[0] if case["norm"] else None, "kw": weight[1] if case["norm"] else None,
            "pos": pos, "inv": inv, "axis": axis}


def _pages(case, g, lead, blocks):
    """Compressed pages [*lead, blocks, hk, page bytes] of random vectors: coordinates of a random
    direction quantized, lognormal norms, residual norms of the codec's own distortion."""
    kb, qjl, vb = _codec(case)
    d, P, H = case["d"], case["page"], case["hk"]
    fields, size = _fields(case)
    pages = torch.zeros((blocks, H, size), dtype=torch.uint8, device="cuda")
    at = {name: (off, n) for name, off, n in fields}
    step = max(1, (1 << 25) // (H * P * d))
    for b0 in range(0, blocks, step):
        nb = min(step, blocks - b0)
        put = {}
        norm = torch.exp(0.3 * torch.randn((nb, H, P), generator=g, device="cuda")) * math.sqrt(d)
        for name, bits in (("kc", kb), ("vc", vb)):
            u = torch.randn((nb, H, P, d), generator=g, device="cuda") / math.sqrt(d)
            if bits == 8:
                put[name] = (u * math.sqrt(d)).to(torch.float8_e4m3fn).view(torch.uint8)
                continue
            mag = _magnitudes(d, bits)
            edge = (0.5 * (mag[1:] + mag[:-1])).float().cuda()
            code = torch.bucketize(u.abs(), edge).to(torch.uint8) | ((u < 0).to(torch.uint8) << (bits - 1))
            per = 8 // bits
            code = code.view(nb, H, P, d // per, per)
            put[name] = functools.reduce(torch.bitwise_or, [code[..., j] << (j * bits) for j in range(per)])
        if qjl:
            put["ks"] = torch.randint(0, 256, (nb, H, P, d // 8), generator=g, device="cuda", dtype=torch.uint8)
            left = {2: 0.342, 4: 0.097}[kb]
            put["kr"] = (left * norm).to(torch.float16).view(torch.uint8).view(nb, H, P, 2)
        put["kn"] = norm.to(torch.float16).view(torch.uint8).view(nb, H, P, 2)
        put["vn"] = norm.flip(-1).to(torch.float16).contiguous().view(torch.uint8).view(nb, H, P, 2)
        for name, v in put.items():
            off, n = at[name]
            pages[b0:b0 + nb, :, off:off + P * n] = v.reshape(nb, H, P * n)
    return pages


def _cross_inputs(case, seed):
    g = _generator(seed)
    ql, kl = _cross_lens(case)
    per = max(1, -(-case["maxkv"] // case["page"]))
    blocks = case["b"] * per
    cache = _pages(case, g, (), blocks)
    table = torch.randperm(blocks, generator=g, device="cuda").view(case["b"], per).to(torch.int32)
    Q = torch.randn((sum(ql), case["hq"], case["d"]), generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0] + list(np.cumsum(ql)), dtype=torch.int32, device="cuda")
    return {"Q": Q, "cu": cu, "table": table, "lens": torch.tensor(kl, dtype=torch.int32, device="cuda"), "cache": cache}


def _pool_inputs(case, seed, lens, children):
    """A pool whose first rows hold pages in random places, and empty rows for the children."""
    g = _generator(seed)
    P, nb = case["page"], case["blocks"]
    caches = torch.randint(0, 256, (case["layers"], nb, case["hk"], _fields(case)[1]), generator=g, device="cuda",
                           dtype=torch.uint8)
    order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    width = -(-max(lens) // P) + 2
    table = torch.full((len(lens) + children, width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(lens):
        k = -(-n // P)
        table[r, :k] = order[at:at + k]
        at += k
    refs[order[:at].long()] = 1
    return {"caches": caches, "refs": refs, "table": table,
            "lens": torch.tensor(lens + [0] * children, dtype=torch.int32, device="cuda")}


def _rows(ids):
    return torch.tensor(ids, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    st = {"case": dict(case)}
    op = case["op"]
    if op == "rope":
        st |= _rope_inputs(case, seed)
        n, hq, hk = case["n"], case["hq"], case["hk"]
        st["q"], st["k"] = st["qkv"][:, :hq], st["qkv"][:, hq:hq + hk]
        st["q_out"] = torch.empty((n, hq, case["d"]), dtype=st["qkv"].dtype, device="cuda")
        st["k_out"] = torch.empty((n, hk, case["d"]), dtype=st["qkv"].dtype, device="cuda")
        if own:
            from kv_cache_vector_07_b200 import tqkv
            st["desc"] = tqkv.rope_desc(case["d"], case["rot"], {"half": tqkv.TQ_ROPE_HALF, "pairs": tqkv.TQ_ROPE_PAIRS}[case["style"]],
                                        pair_axis=st["axis"], n_axes=case["axes"], eps=1e-6)
        return st
    kb, qjl, vb = _codec(case)
    if own:
        from kv_cache_vector_07_b200 import tqkv
        st["desc"] = tqkv.cache_desc(case["d"], kb, qjl, vb, page_tokens=case["page"], n_kv_heads=case["hk"])
    if op == "cross":
        st |= _cross_inputs(case, seed)
        st["out"] = torch.zeros_like(st["Q"])
        if own:
            st["kp"], st["vp"] = _handles(case["d"], kb, vb)
            st["ws"] = torch.zeros(tqkv.cross_workspace_bytes(st["desc"], case["b"], st["Q"].shape[0], case["maxq"], case["hq"],
                                                              case["maxkv"]), dtype=torch.uint8, device="cuda")
        return st
    if op == "fork":
        lens = _lens(case, "plen", case["parents"], case["plen"], False)
        kids = case["parents"] * case["each"]
        st |= _pool_inputs(case, seed, lens, kids)
        st["src"] = _rows([i // case["each"] for i in range(kids)])
        st["dst"] = _rows([len(lens) + i for i in range(kids)])
        new = [0] * len(lens) + [case["new"]] * kids
        st["new"] = _rows(new)
        st["slots"] = torch.zeros(sum(new), dtype=torch.int32, device="cuda")
    else:
        lens, kept, sink = _evict_lens(case)
        st |= _pool_inputs(case, seed, lens, len(lens))
        r = np.random.default_rng(seed)
        keep = np.zeros((len(lens), max(kept)), np.int32)
        for i, (n, k, s) in enumerate(zip(lens, kept, sink)):
            keep[i, :s] = np.arange(s)
            keep[i, s:k] = s + np.sort(r.permutation(n - s)[:k - s])
        st["keep"], st["kept"] = torch.from_numpy(keep).cuda(), _rows(kept)
        st["src"] = _rows(list(range(len(lens))))
        st["dst"] = _rows([len(lens) + i for i in range(len(lens))])
    if own:
        st["layers"] = list(st["caches"].unbind(0))
        st["ws"] = torch.zeros(tqkv.pages_workspace_bytes(case["blocks"], *st["table"].shape), dtype=torch.uint8, device="cuda")
    return st


@functools.lru_cache(maxsize=None)
def _handles(d, kb, vb):
    from kv_cache_vector_07_b200 import tqkv
    return tqkv.make_params(d, kb, 1001), tqkv.make_params(d, vb, 2001)


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        from kv_cache_vector_07_b200 import tqkv
        if op == "rope":
            return tqkv.qk_norm_rope(st["desc"], st["q"], st["k"], st["pos"], st["inv"], q_weight=st["qw"], k_weight=st["kw"],
                                     q_out=st["q_out"], k_out=st["k_out"])
        if op == "cross":
            return tqkv.cross_attn(st["kp"], st["vp"], st["desc"], st["Q"], st["cu"], st["case"]["maxq"], st["table"], st["lens"],
                                   st["case"]["maxkv"], st["cache"], out=st["out"], workspace=st["ws"])
        tqkv.pages_fork(st["desc"], st["layers"], st["refs"], st["table"], st["lens"], st["src"], st["dst"], workspace=st["ws"])
        if op == "fork":
            tqkv.pages_reserve(st["desc"], st["refs"], st["table"], st["lens"], st["new"], st["slots"], workspace=st["ws"])
        else:
            tqkv.pages_compact(st["desc"], st["layers"], st["refs"], st["table"], st["lens"], st["dst"], st["keep"], st["kept"],
                               workspace=st["ws"])
        tqkv.pages_free(st["desc"], st["refs"], st["table"], st["lens"], st["dst"], workspace=st["ws"])
    else:
        if op == "rope":
            return [_plain_rope(st, st["q"], st["qw"]), _plain_rope(st, st["k"], st["kw"])]
        if op == "cross":
            return _plain_cross(st)
        _plain_fork(st)
        if op == "fork":
            _plain_reserve(st)
        else:
            _plain_compact(st)
        _plain_free(st)
    got = [st["table"], st["lens"], st["refs"], st["caches"]]
    return got + [st["slots"]] if op == "fork" else got


def _plain_rope(st, x, weight):
    c = st["case"]
    rot, h = c["rot"], c["rot"] // 2
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    axis = torch.tensor(st["axis"], device="cuda")
    ang = st["pos"].double()[axis].t() * st["inv"].double()      # [n, pairs]; far positions need the 64 bits
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    out = y.clone()
    if c["style"] == "half":
        a, b = y[..., :h], y[..., h:rot]
        out[..., :h], out[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def _plain_codes(raw, bits, d, mag):
    """Levels [.., d] of packed sign-magnitude codes [.., bytes]."""
    shift = torch.arange(0, 8, bits, device="cuda", dtype=torch.uint8)
    code = ((raw[..., None] >> shift) & ((1 << bits) - 1)).flatten(-2).long()
    return torch.cat([mag, -mag])[code]


def _plain_cross(st):
    c = st["case"]
    kb, qjl, vb = _codec(c)
    d, P, H, B = c["d"], c["page"], c["hk"], c["b"]
    G, maxq, maxkv = c["hq"] // H, c["maxq"], c["maxkv"]
    had = _hadamard(d, "cuda", torch.float32) / math.sqrt(d)
    pages = st["cache"][st["table"].long()].transpose(1, 2)                      # [B, H, blocks, bytes]
    f = {name: pages[..., off:off + P * n].reshape(B, H, -1, n)[:, :, :maxkv] for name, off, n in _fields(c)[0]}
    half = lambda name: f[name].contiguous().view(torch.float16).float()  # noqa: E731
    if kb == 8:
        k = half("kn") * f["kc"].contiguous().view(torch.float8_e4m3fn).float() / math.sqrt(d)
    else:
        k = half("kn") * _plain_codes(f["kc"], kb, d, _magnitudes(d, kb).float().cuda())
    if qjl:
        s = 2 * ((f["ks"][..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1).flatten(-2).float() - 1
        k = k + half("kr") * (math.sqrt(math.pi / 2) / d) * (s @ _projection(d, 1001).float().cuda())
    v = half("vn") * _plain_codes(f["vc"], vb, d, _magnitudes(d, vb).float().cuda())
    # the runs padded to the longest: [B, H, G maxq, d]
    ql = (st["cu"][1:] - st["cu"][:-1]).long()
    j = torch.arange(maxq, device="cuda")
    there = j[None] < ql[:, None]
    at = (st["cu"][:-1].long()[:, None] + j[None])[there]
    q = torch.zeros((B, maxq, c["hq"], d), device="cuda")
    q[there] = st["Q"].float()[at]
    q = ((q * _signs(d, 1001).float().cuda()) @ had.t()).view(B, maxq, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * maxq, d)
    s = q @ k.transpose(-1, -2) / math.sqrt(d)
    s.masked_fill_((torch.arange(maxkv, device="cuda") >= st["lens"][:, None])[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    o = (o @ had) * _signs(d, 2001).float().cuda()
    o = o.view(B, H, G, maxq, d).permute(0, 3, 1, 2, 4).reshape(B, maxq, c["hq"], d)
    out = torch.zeros_like(st["Q"])
    out[at] = o[there].to(torch.bfloat16)
    return out


def _plain_take(st, need):
    """Lowest free pages, dealt in the order of the requests: [need.sum()] ids, marked as taken."""
    ids = torch.nonzero(st["refs"] == 0).flatten()[:int(need.sum())]
    st["refs"][ids] = 1
    return ids.to(torch.int32)


def _plain_fork(st):
    P = st["case"]["page"]
    src, dst, table, lens = st["src"].long(), st["dst"].long(), st["table"], st["lens"]
    n = lens[src].long()
    full, part = n // P, n % P != 0
    col = torch.arange(table.shape[1], device="cuda")
    shared = col[None] < full[:, None]
    rows = table[src]
    st["refs"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    fresh = _plain_take(st, part)
    old = rows[part, full[part]].long()
    rows[part, full[part]] = fresh
    table[dst] = torch.where(col[None] < (full + part)[:, None], rows, table[dst])
    lens[dst] = n.to(torch.int32)
    st["caches"][:, fresh.long()] = st["caches"][:, old]


def _plain_reserve(st):
    P = st["case"]["page"]
    table, lens, new = st["table"], st["lens"].long(), st["new"].long()
    have, want = (lens + P - 1) // P, (lens + new + P - 1) // P
    col = torch.arange(table.shape[1], device="cuda")
    put = (col[None] >= have[:, None]) & (col[None] < want[:, None])
    table[put] = _plain_take(st, want - have)
    row = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new)
    pos = lens[row] + torch.arange(len(row), device="cuda") - (torch.cumsum(new, 0) - new)[row]
    st["slots"].copy_(table[row, pos // P].long() * P + pos % P)
    st["lens"] += st["new"]


def _plain_compact(st):
    c = st["case"]
    P = c["page"]
    rows, table, lens, keep, kept = st["dst"].long(), st["table"], st["lens"], st["keep"].long(), st["kept"].long()
    old = table[rows]                                                            # [R, width]
    width = table.shape[1]
    had, want = (lens[rows].long() + P - 1) // P, (kept + P - 1) // P
    col = torch.arange(width, device="cuda")
    pos = torch.arange(width * P, device="cuda")
    k = torch.nn.functional.pad(keep, (0, max(0, width * P - keep.shape[1])))[:, :width * P]
    same = ((k == pos[None]) | (pos[None] >= kept[:, None])).view(len(rows), width, P).all(-1)
    alone = st["refs"][old.clamp(min=0).long()] == 1
    used = col[None] < want[:, None]
    stay = used & same & (((col + 1) * P)[None].le(kept[:, None]) | alone)
    fresh = used & ~stay
    ids = _plain_take(st, fresh.sum(1))
    now = old.clone()
    now[fresh] = ids
    gone = (col[None] < had[:, None]) & ~stay
    st["refs"].index_add_(0, old[gone].long(), -torch.ones_like(old[gone]))
    table[rows] = torch.where(used, now, table[rows])
    lens[rows] = kept.to(torch.int32)
    move = (pos[None] < kept[:, None]) & fresh.repeat_interleave(P, 1)
    r, p = torch.nonzero(move, as_tuple=True)
    frm, to, tok = old[r, k[r, p] // P].long(), now[r, p // P].long(), k[r, p] % P
    caches = st["caches"]
    for _, off, n in _fields(c)[0]:
        view = caches[..., off:off + P * n].unflatten(-1, (P, n))                # [layers, blocks, H, P, n]
        view[:, to, :, p % P] = view[:, frm, :, tok]


def _plain_free(st):
    P = st["case"]["page"]
    rows = st["dst"].long()
    col = torch.arange(st["table"].shape[1], device="cuda")
    ids = st["table"][rows][col[None] < ((st["lens"][rows].long() + P - 1) // P)[:, None]].long()
    st["refs"].index_add_(0, ids, -torch.ones_like(ids, dtype=torch.int32))
    st["lens"][rows] = 0


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "rope":
        return _exact_rope(case, _rope_inputs(case, seed))
    if case["op"] == "cross":
        return _exact_cross(case, _cross_inputs(case, seed))
    return None                                              # bytes and tables: no computed numbers


def _exact_rope(case, x):
    got = []
    for lo, n, weight in ((0, case["hq"], x["qw"]), (case["hq"], case["hk"], x["kw"])):
        v = x["qkv"][:, lo:lo + n].to(torch.float64)
        if weight is not None:
            v = v / (v.pow(2).sum(-1, keepdim=True) / case["d"] + float(np.float32(1e-6))).sqrt() * weight.to(torch.float64)
        turn = torch.stack([x["pos"][a].to(torch.float64) * f for a, f in zip(x["axis"], x["inv"].to(torch.float64))], 1)
        e = torch.polar(torch.ones_like(turn), turn)[:, None]    # e^(i angle) for every token and pair
        head, tail = v[..., :case["rot"]], v[..., case["rot"]:]
        if case["style"] == "half":
            z = torch.complex(*[t.contiguous() for t in head.chunk(2, -1)]) * e
            head = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * e
            head = torch.view_as_real(z).flatten(-2)
        got.append(torch.cat([head, tail], -1))
    return got


def _exact_cross(case, x):
    kb, qjl, vb = _codec(case)
    d, P, H = case["d"], case["page"], case["hk"]
    G = case["hq"] // H
    f64 = torch.float64
    at = {name: (off, n) for name, off, n in _fields(case)[0]}
    R = [_hadamard(d, "cuda", f64) * _signs(d, s).cuda()[None] / math.sqrt(d) for s in (1001, 2001)]   # y = R x
    ql, kl = _cross_lens(case)
    out = torch.zeros(x["Q"].shape, dtype=f64, device="cuda")
    begin = 0
    for b in range(case["b"]):
        if ql[b] and kl[b]:
            ids = x["table"][b, :-(-kl[b] // P)].long()
            for h in range(H):
                def field(name):
                    off, n = at[name]
                    return x["cache"][ids, h, off:off + P * n].reshape(-1, n)[:kl[b]]

                def number(name):
                    return field(name).contiguous().view(torch.float16).to(f64)

                def levels(name, bits):
                    raw = field(name)
                    bit = torch.stack([(raw >> i) & 1 for i in range(8)], -1).flatten(1).view(len(raw), d, bits).to(torch.int64)
                    rank = sum(bit[..., i] << i for i in range(bits - 1)) if bits > 1 else torch.zeros_like(bit[..., 0])
                    return _magnitudes(d, bits).cuda()[rank] * (1 - 2 * bit[..., bits - 1]).to(f64)

                if kb == 8:
                    key = field("kc").contiguous().view(torch.float8_e4m3fn).to(f64) / math.sqrt(d) * number("kn")
                else:
                    key = levels("kc", kb) * number("kn")
                if qjl:
                    raw = field("ks")
                    bit = torch.stack([(raw >> i) & 1 for i in range(8)], -1).flatten(1).to(f64)
                    key = key + number("kr") * math.sqrt(math.pi / 2) / d * ((bit - (1 - bit)) @ _projection(d, 1001).cuda())
                key, val = key @ R[0], (levels("vc", vb) * number("vn")) @ R[1]  # back in the vectors' own coordinates
                q = x["Q"][begin:begin + ql[b], h * G:(h + 1) * G].to(f64)
                p = torch.softmax(torch.einsum("qgd,kd->qgk", q, key) / math.sqrt(d), -1)
                out[begin:begin + ql[b], h * G:(h + 1) * G] = torch.einsum("qgk,kd->qgd", p, val)
        begin += ql[b]
    return out
