"""tq_cross_attn against its formula in 64 bits, on the bytes that the cache holds.

The reference decodes the pages with the oracle's layout and evaluates the formula with numpy
(it equals the oracle's attention, test_reference_is_the_oracles_attention).

Tolerances count roundings.  Products may be taken with keys, values, queries and softmax
weights rounded to fp16 (half a step, u = 2^-11, each) and summed in fp32 (at most d + 16
half steps of 2^-24 on a logit), so logit t is off by at most
    delta_t = (2 u + u^2 + (d + 16) 2^-24) sum_i |(R q)_i k_t,i| / sqrt(d) + 2^-22 |l_t| + 2^-20
(the last two: exponents in base 2 and the exponential's own error), every weight by a factor
within exp(+-(delta_t + sum_t p_t delta_t)), and a rotated output coordinate by
    sum_t p_t |v_t| (expm1(delta_t + mean delta) + 2 u + u^2 + 2^-18);
the inverse rotation spreads that with |R|, and the result is rounded to bf16 once (half a
step, 2^-8).  On top, the errors must not pile up at their bound: over a whole call their
2-norm stays under 2^-8 of the result's (a bf16 rounding alone gives about 2^-9.2).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import parity
from kv_cache_vector_07_b200 import synth, tqkv
from oracle import oracle as O

DEV = "cuda"
U = 2.0 ** -11


class Codec:
    """Library and oracle parameters of one cache."""

    def __init__(self, d, kbits, kqjl, vbits, P=64, H=1, dense=False, seed=3):
        lib = lambda b: tqkv.TQ_BITS_POLAR if b == "polar" else (tqkv.half_bits(b) if b != int(b) else int(b))
        rot, orot = (tqkv.TQ_ROT_DENSE, "dense") if dense else (tqkv.TQ_ROT_HADAMARD, "hadamard")
        ora = lambda b, s: O.polar_params(d, s, rotation=orot) if b == "polar" else O.make_params(d, b, s, rotation=orot)
        self.d, self.kbits, self.kqjl, self.vbits, self.P, self.H = d, kbits, kqjl, vbits, P, H
        self.lay = O.Layout(d, kbits, kqjl, vbits, page_tokens=P)
        self.Pk, self.Pv = ora(kbits, 1000 + seed), ora(vbits, 2000 + seed)
        self.R = [O.rotate(np.eye(d), p.signs, p.Rm).T for p in (self.Pk, self.Pv)]          # y = R x
        if torch.cuda.is_available():
            self.desc = tqkv.cache_desc(d, lib(kbits), kqjl, lib(vbits), page_tokens=P, n_kv_heads=H)
            self.kp, self.vp = tqkv.make_params(d, lib(kbits), 1000 + seed, rot), tqkv.make_params(d, lib(vbits), 2000 + seed, rot)

    def _levels(self, bits, P, idx, n):
        if bits == "polar":
            return O.polar_decode(idx[0], idx[1], n, P)
        if bits == 8:
            return np.array([O.e4m3_value(c) for c in range(256)])[idx] / math.sqrt(self.d) * n[:, None]
        return parity.levels_of(P, idx) * n[:, None]

    def states(self, cache, slots, head):
        """Keys and values of the slots in their rotated bases, 64 bits."""
        f = O.read_cache(self.lay, cache, slots, head, self.H)
        k = self._levels(self.kbits, self.Pk, f["kidx"], f["kn"])
        if self.kqjl:
            k = k + f["kr"][:, None] * math.sqrt(math.pi / 2) / self.d * ((2.0 * f["ks"] - 1) @ self.Pk.S.astype(np.float64))
        return k, self._levels(self.vbits, self.Pv, f["vidx"], f["vn"])

    def attend(self, Q, k, v):
        """(out, lse, tolerance of out, tolerance of lse) of queries Q [n, d]."""
        d = self.d
        if not len(k):
            z = np.zeros(len(Q))
            return np.zeros((len(Q), d)), z - np.inf, np.zeros((len(Q), d)), z
        q = Q @ self.R[0].T
        s = q @ k.T / math.sqrt(d)
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(1, keepdims=True)
        p /= total
        delta = (2 * U + U * U + (d + 16) * 2.0 ** -24) * (np.abs(q) @ np.abs(k).T) / math.sqrt(d) + 2.0 ** -22 * np.abs(s) + 2.0 ** -20
        mean = (p * delta).sum(1, keepdims=True)
        off = (p * (np.expm1(delta + mean) + 2 * U + U * U + 2.0 ** -18)) @ np.abs(v)
        out = p @ v @ self.R[1]
        tol = off @ np.abs(self.R[1])
        tol = tol + 2.0 ** -8 * (np.abs(out) + tol) + 2.0 ** -130
        lse = (top + np.log(total))[:, 0]
        return out, lse, tol, mean[:, 0] * 1.01 + 2.0 ** -20 * (1 + np.abs(lse))


class Call:
    """Random states in a shuffled cache and ragged runs of queries."""

    def __init__(self, cd, qlens, kvlens, G, seed=0, extra_rows=0, scale=1.0):
        self.cd, self.qlens, self.kvlens, self.G = cd, qlens, kvlens, G
        d, H, P, B = cd.d, cd.H, cd.P, len(kvlens)
        self.maxkv = max(kvlens + [0])
        width = max(1, -(-self.maxkv // P))
        blocks = B * width + 3
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(blocks, generator=g)[:B * width].view(B, width).to(torch.int32)
        self.cache = tqkv.alloc_cache(cd.desc, blocks)
        self.cache.random_(0, 256)                                   # what lies behind a sequence is not read
        slots, n = [], sum(kvlens)
        for b, L in enumerate(kvlens):
            pos = torch.arange(L)
            slots.append(self.table[b].long()[pos // P] * P + pos % P)
        self.slots = [s.numpy().astype(np.int32) for s in slots]
        if n:
            K = synth.outlier_normal((n, H, d), seed=seed + 1, device=DEV) * scale
            V = synth.outlier_normal((n, H, d), seed=seed + 2, device=DEV, channels=(3,), scale=8.0)
            tqkv.encode(cd.kp, cd.vp, cd.desc, K.contiguous(), V, torch.cat(slots).to(torch.int32).to(DEV), self.cache)
        self.total = sum(qlens) + extra_rows
        self.Q = synth.normal((self.total, G * H, d), seed=seed + 3, device=DEV)
        self.cu = torch.tensor([0] + list(np.cumsum(qlens)), dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(kvlens, dtype=torch.int32, device=DEV)
        self.table = self.table.to(DEV)
        self.args = (cd.kp, cd.vp, cd.desc, self.Q, self.cu, max(qlens + [0]), self.table, self.lens, self.maxkv, self.cache)

    def run(self, **kw):
        out = torch.full_like(self.Q, 7.0)
        lse = torch.full(self.Q.shape[:2], 7.0, device=DEV)
        ws = torch.zeros(tqkv.cross_workspace_bytes(self.cd.desc, len(self.kvlens), self.total, self.args[5], self.Q.shape[1],
                                                    self.maxkv), dtype=torch.uint8, device=DEV)
        tqkv.cross_attn(*self.args, out=out, lse=lse, workspace=ws, **kw)
        torch.cuda.synchronize()
        return out, lse, tqkv.read_status(ws)

    def reference(self, rows=None, missing=None):
        """Per sequence: (row indices, head h's slice, out, lse, tolerances); missing: {b: mask of keys left out}."""
        raw = self.cache.view(self.cache.shape[0] * self.cd.H, -1).cpu().numpy()
        Q = self.Q.double().cpu().numpy()
        at = 0
        for b, n in enumerate(self.qlens):
            if n:
                pick = np.arange(at, at + n) if rows is None else at + np.unique(np.clip(rows, 0, n - 1))
                for h in range(self.cd.H):
                    k, v = self.cd.states(raw, self.slots[b], h)
                    if missing and b in missing:
                        k, v = k[~missing[b]], v[~missing[b]]
                    hs = slice(h * self.G, (h + 1) * self.G)
                    got = self.cd.attend(Q[pick, hs].reshape(-1, self.cd.d), k, v)
                    yield (pick, hs, *got)
            at += n

    def check(self, out, lse, **kw):
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        err2 = ref2 = 0.0
        for pick, hs, ref, rl, tol, tl in self.reference(**kw):
            e = np.abs(o[pick, hs].reshape(ref.shape) - ref)
            assert (e <= tol).all(), f"out: {(e > tol).sum()} of {e.size} off, worst {(e / np.maximum(tol, 1e-300)).max():.3g} tolerances"
            g = l[pick, hs].reshape(-1)
            assert np.array_equal(np.isinf(g), np.isinf(rl)) and np.array_equal(g[np.isinf(rl)], rl[np.isinf(rl)])
            f = np.isfinite(rl)
            assert (np.abs(g[f] - rl[f]) <= tl[f]).all(), np.abs(g[f] - rl[f]).max()
            err2, ref2 = err2 + (e ** 2).sum(), ref2 + (ref ** 2).sum()
        assert err2 <= 2.0 ** -16 * ref2, math.sqrt(err2 / ref2)
        used = sum(self.qlens)
        assert (out[used:] == 7).all() and (lse[used:] == 7).all()


CODECS = {
    "k3v4": (128, 2, True, 4), "k5v4": (128, 4, True, 4), "k8v4": (128, 8, False, 4), "33": (128, 3, False, 3),
    "11": (128, 1, True, 1), "frac": (128, 2.5, True, 3.5), "polar": (128, "polar", True, "polar"), "k3v2": (128, 3, True, 2),
    "d64": (64, 2, True, 4), "d64k8": (64, 8, False, 4), "d64frac": (64, 1.5, True, 2.5), "d64polar": (64, "polar", False, "polar"),
    "d32": (32, 4, True, 4), "d256": (256, 4, True, 3), "d8": (8, 2, True, 2),
}
CASES = [
    # codec, P, H, G, query lengths, state lengths, rows behind the last run
    ("k3v4", 64, 2, 4, [1, 1, 1], [70, 1, 64], 0),
    ("k3v4", 64, 2, 4, [100, 3, 0, 300], [700, 129, 5, 128], 2),
    ("k5v4", 64, 1, 8, [65, 40], [1000, 333], 0),
    ("k5v4", 16, 3, 3, [43, 200, 1], [127, 515, 2], 5),
    ("k8v4", 8, 1, 5, [77, 50], [300, 1], 0),
    ("33", 24, 2, 1, [130, 257, 5], [65, 640, 0], 1),
    ("11", 64, 1, 2, [80], [2049], 0),
    ("frac", 64, 1, 4, [64, 33], [256, 100], 0),
    ("polar", 32, 1, 2, [90], [400], 0),
    ("k3v2", 256, 1, 6, [50, 50], [257, 1000], 0),
    ("d64", 64, 2, 4, [100, 9], [900, 31], 0),
    ("d64", 64, 1, 7, [33, 1, 0, 60], [200, 0, 9, 1501], 0),
    ("d64k8", 16, 2, 5, [333, 7], [1501, 1], 3),
    ("d64frac", 64, 1, 2, [70], [130], 0),
    ("d64polar", 64, 1, 2, [70], [130], 0),
    ("d32", 64, 2, 2, [40, 3], [300, 64], 0),
    ("d256", 64, 1, 2, [40, 3], [150, 64], 0),
    ("d8", 8, 2, 3, [20, 1], [90, 0], 1),
    ("k3v4", 64, 8, 4, [2, 5, 1, 1], [4000, 33, 64, 1], 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("codec,P,H,G,qlens,kvlens,extra", CASES)
def test_values(codec, P, H, G, qlens, kvlens, extra):
    c = Call(Codec(*CODECS[codec], P=P, H=H), qlens, kvlens, G, seed=len(qlens) + G, extra_rows=extra)
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse)


@pytest.mark.gpu
def test_dense_rotation():
    c = Call(Codec(128, 4, True, 4, H=2, dense=True), [70, 5], [300, 64], 2)
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("codec", ["k5v4", "d64k8"])
def test_long_states_few_rows(codec):
    """The key axis is split where there are few rows; sampled rows of a longer run too."""
    cd = Codec(*CODECS[codec], H=2)
    for qlens in ([40], [3, 150]):
        c = Call(cd, qlens, [9000] * len(qlens), 2, seed=5)
        out, lse, flags = c.run()
        assert flags == 0
        c.check(out, lse, rows=[0, 1, 2, 77, 149])


@pytest.mark.gpu
def test_rows_behind_the_runs_of_a_split_call():
    """The key axis is split and Q has many rows that belong to no run."""
    c = Call(Codec(*CODECS["k5v4"], H=1), [30, 7], [5000, 3000], 4, seed=8, extra_rows=500)
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse)


@pytest.mark.gpu
def test_more_queries_than_one_round_by_rows():
    """Head sizes that go by rows take 65,536 rows of a head at once."""
    c = Call(Codec(*CODECS["d32"], H=8), [900, 600], [100, 64], 8, extra_rows=40)
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse, rows=[0, 1, 500, 599, 899])


@pytest.mark.gpu
def test_more_states_than_one_round_holds():
    """528 pairs of 64 tiles of 32 KB: the operand tiles take two rounds."""
    kv = [8192] + [64] * 63 + [8190, 300]
    c = Call(Codec(*CODECS["d64"], H=8), [7] + [0] * 62 + [2, 5, 9], kv, 1, seed=4)
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse, rows=[0, 4, 8])


@pytest.mark.gpu
def test_two_calls_at_once():
    """On two streams, with a workspace each."""
    calls = [Call(Codec(*CODECS[n], H=2), [200, 90], [900, 1500], 4, seed=i) for i, n in enumerate(("k5v4", "k3v4"))]
    want = [c.run()[0] for c in calls]
    got = [torch.zeros_like(w) for w in want]
    ws = [torch.zeros(tqkv.cross_workspace_bytes(c.cd.desc, 2, c.total, 200, 8, 1500), dtype=torch.uint8, device=DEV) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, o, w, st in zip(calls, got, ws, streams):
            tqkv.cross_attn(*c.args, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("codec", ["k5v4", "k3v4"])
@pytest.mark.parametrize("as_number", [False, True])
def test_what_the_call_makes_belongs_to_its_stream(codec, as_number):
    """out and workspace not given, the current stream busy: what clears them
    must not come behind the call's own kernels."""
    c = Call(Codec(*CODECS[codec], H=2), [3, 1] if codec == "k3v4" else [70, 9], [300, 500], 4)
    want = c.run()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)
    for _ in range(40):                                              # some milliseconds of work
        busy += 1
    got = tqkv.cross_attn(*c.args, stream=side.cuda_stream if as_number else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
def test_any_number_out_of_range_is_reported(page):
    for qlens in ([2, 1], [70, 40]):
        c = Call(Codec(*CODECS["k3v4"], H=2), qlens, [300, 200], 2)
        c.table[1, 3] = page                                         # tokens 192 .. 199
        out, lse, flags = c.run()
        assert flags == tqkv.TQ_DEV_BLOCK_RANGE
        c.check(out, lse, missing={1: np.arange(200) >= 192})


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** -12, 2.0 ** 8])
def test_small_and_large_states(scale):
    c = Call(Codec(*CODECS["k5v4"], H=1), [70], [500], 4, scale=scale)
    c.Q /= 16 * scale
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("qlens", [[2, 1], [70, 40]])
def test_missing_pages_short_runs_and_long_lengths(qlens):
    cd = Codec(*CODECS["k3v4"], H=2)
    c = Call(cd, qlens, [300, 200], 2)
    c.table[0, 2] = -1                                               # tokens 128 .. 191 of sequence 0
    c.table[1, 0] = c.cache.shape[0]                                 # tokens 0 .. 63 of sequence 1
    out, lse, flags = c.run()
    assert flags == tqkv.TQ_DEV_BLOCK_RANGE
    gone = [np.arange(300) // 64 == 2, np.arange(200) // 64 == 0]
    c.check(out, lse, missing=dict(enumerate(gone)))
    # every page of a sequence missing: as an empty one
    c.table[1] = -7
    out, lse, flags = c.run()
    assert flags == tqkv.TQ_DEV_BLOCK_RANGE
    c.check(out, lse, missing={0: gone[0], 1: np.ones(200, bool)})


@pytest.mark.gpu
@pytest.mark.parametrize("qlens", [[2, 1], [70, 40]])
def test_long_lengths_end_at_the_most_and_long_runs_are_cut(qlens):
    c = Call(Codec(*CODECS["k3v4"], H=2), qlens, [300, 300], 2)
    first, _, flags = c.run()
    c.lens += 5000
    out, lse, more = c.run()
    assert flags == more == 0 and torch.equal(out, first)
    n = qlens[0]
    c.args = c.args[:5] + (n - 1,) + c.args[6:]
    out, lse, flags = c.run()
    assert flags == tqkv.TQ_DEV_ROW
    assert (out[n - 1] == 7).all() and (lse[n - 1] == 7).all()
    c.check(out, lse, rows=list(range(n - 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("qlens", [[1, 1], [90, 64]])
def test_non_finite_query_rows_stay_alone(qlens):
    c = Call(Codec(*CODECS["k3v4"], H=1), qlens, [100, 300], 2)
    ref, _, _ = c.run()
    bad = sum(qlens) - 1
    c.Q[bad, 0, 5], c.Q[bad, 1, 9] = float("nan"), float("inf")
    out, lse, _ = c.run()
    assert torch.equal(out[:bad], ref[:bad]) and torch.isnan(out[bad, :2]).all() and torch.isnan(lse[bad, :2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("qlens", [[1, 1, 1], [100, 60, 7]])
def test_same_bits_every_time_on_another_stream_and_in_a_graph(qlens):
    c = Call(Codec(*CODECS["k5v4"], H=2), qlens, [700, 90, 1], 4)
    out, lse, _ = c.run()
    for _ in range(3):
        again, l2, _ = c.run()
        assert torch.equal(again, out) and torch.equal(l2, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(tqkv.cross_workspace_bytes(c.cd.desc, 3, c.total, max(qlens), 8, 700), dtype=torch.uint8, device=DEV)
    other = torch.zeros_like(out)
    torch.cuda.synchronize()
    tqkv.cross_attn(*c.args, out=other, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tqkv.cross_attn(*c.args, out=other, workspace=ws)
    c.lens.copy_(torch.tensor([333, 64, 0]))                          # read at replay
    want, _, _ = c.run()
    other.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, want) and (want[sum(qlens[:2]):] == 0).all()


def test_reference_is_the_oracles_attention():
    r = np.random.default_rng(0)
    for d, kb, qjl, vb in ((64, 2, True, 4), (64, 8, False, 3), (32, "polar", True, "polar"), (32, 2.5, True, 1.5)):
        cd = Codec(d, kb, qjl, vb, P=16)
        enc = lambda P, b, x, q: O.encode_polar(x, P, qjl=q) if b == "polar" else O.encode(x, P, qjl=q)
        Ek, Ev = enc(cd.Pk, kb, r.standard_normal((50, d)), qjl), enc(cd.Pv, vb, r.standard_normal((50, d)), False)
        cache = np.zeros((4, cd.lay.page_bytes), np.uint8)
        slots = np.arange(50, dtype=np.int32)
        O.write_cache(cd.lay, cache, slots, 0, 1, Ek, Ev)
        Q = r.standard_normal((6, d))
        out, lse, _ = O.attend(Q, cd.Pk, Ek, cd.Pv, Ev)
        got = cd.attend(Q, *cd.states(cache, slots, 0))
        assert np.allclose(got[0], out, rtol=0, atol=1e-9) and np.allclose(got[1], lse, rtol=0, atol=1e-9)


class _FakeParams(ctypes.Structure):
    """The first fields of a parameter handle (never followed further by a refusal)."""
    _fields_ = [("d", ctypes.c_int), ("bits", ctypes.c_int)]


def _c(desc=None, k=(128, 2), v=(128, 4), Q=256, total=8, max_q=4, Hq=4, cu=256, B=2, table=256, width=4, lens=256, maxkv=256,
       cache=256, out=256, lse=None, ws=256, ws_bytes=1 << 40):
    desc = tqkv.cache_desc(128, 2, True, 4, n_kv_heads=2) if desc is None else desc
    kp, vp = (ctypes.byref(_FakeParams(*x)) if x else None for x in (k, v))
    return tqkv._lib.tq_cross_attn(kp, vp, ctypes.byref(desc), Q, total, max_q, Hq, cu, B, table, width, lens, maxkv, cache, 8,
                                   out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), tqkv.TQ_EINVAL), (dict(v=None), tqkv.TQ_EINVAL), (dict(k=(64, 2)), tqkv.TQ_EINVAL),
    (dict(v=(128, 3)), tqkv.TQ_EINVAL), (dict(desc=tqkv.cache_desc(128, 2, True, 0, n_kv_heads=2)), tqkv.TQ_EINVAL),
    (dict(desc=tqkv.cache_desc(512, 2, True, 4)), tqkv.TQ_EUNSUPPORTED), (dict(Hq=18), tqkv.TQ_EUNSUPPORTED),
    (dict(Hq=3), tqkv.TQ_EINVAL), (dict(Hq=0), tqkv.TQ_EINVAL), (dict(total=-1), tqkv.TQ_EINVAL), (dict(max_q=-1), tqkv.TQ_EINVAL),
    (dict(B=-1), tqkv.TQ_EINVAL), (dict(maxkv=-1), tqkv.TQ_EINVAL), (dict(maxkv=257), tqkv.TQ_EINVAL),
    (dict(total=1 << 30), tqkv.TQ_EINVAL), (dict(maxkv=2 ** 31 - 1, width=1 << 30), tqkv.TQ_EINVAL), (dict(Q=None), tqkv.TQ_EINVAL), (dict(Q=264), tqkv.TQ_EINVAL),
    (dict(cu=None), tqkv.TQ_EINVAL), (dict(table=None), tqkv.TQ_EINVAL), (dict(lens=None), tqkv.TQ_EINVAL),
    (dict(lens=2), tqkv.TQ_EINVAL), (dict(cache=128), tqkv.TQ_EINVAL), (dict(out=None), tqkv.TQ_EINVAL),
    (dict(lse=2), tqkv.TQ_EINVAL), (dict(ws=None), tqkv.TQ_EINVAL), (dict(ws=64), tqkv.TQ_EINVAL)])
def test_c_refusals(kw, code):
    assert _c(**kw) == code


def test_c_nothing_to_do_is_ok():
    for kw in (dict(B=0), dict(total=0), dict(max_q=0)):
        assert _c(**kw, Q=None, out=None) == tqkv.TQ_OK


def test_workspace_bytes():
    desc = tqkv.cache_desc(128, 2, True, 4, n_kv_heads=2)
    f = lambda *a: tqkv.cross_workspace_bytes(desc, *a)
    assert f(-1, 8, 4, 4, 64) == f(2, 8, 4, 3, 64) == f(2, 8, 4, 4, -1) == 0
    assert f(2, 8, 4, 4, 64) <= f(2, 800, 400, 4, 64) <= f(2, 800, 400, 4, 6400)


@pytest.mark.gpu
def test_binding_refusals():
    c = Call(Codec(*CODECS["k3v4"], H=1), [3], [70], 2)
    names = ("kp", "vp", "desc", "Q", "cu_q", "max_q", "block_table", "kv_lens", "max_kv_len", "cache")
    good = dict(zip(names, c.args))
    tqkv.cross_attn(**good)
    for kw in (dict(Q=c.Q.float()), dict(Q=c.Q[..., :64].contiguous()), dict(Q=c.Q.transpose(0, 1)), dict(Q=c.Q.cpu()),
               dict(cu_q=c.cu.long()), dict(cu_q=c.cu[:1]), dict(kv_lens=c.lens.long()), dict(kv_lens=c.lens.view(1, 1)),
               dict(block_table=c.table.view(-1)), dict(block_table=c.table.long()), dict(cache=c.cache[..., :16].contiguous()),
               dict(out=torch.empty((2, 2, 128), device=DEV, dtype=torch.bfloat16)), dict(lse=torch.empty((3, 1), device=DEV)),
               dict(lse=torch.empty((3, 2), device=DEV, dtype=torch.float64))):
        with pytest.raises(ValueError):
            tqkv.cross_attn(**dict(good, **kw))
    with pytest.raises(tqkv.TQError):
        tqkv.cross_attn(**dict(good, workspace=torch.zeros(256, device=DEV, dtype=torch.uint8)))
    with pytest.raises(tqkv.TQError):
        tqkv.cross_attn(**dict(good, max_kv_len=1000))
