"""tq_cross_attn where the sizes of states, values and queries differ: zero states, value norms
that change from tile to tile, strong keys without a value, queries near the end of bf16's range.

Formula, tolerances and their derivation: test_cross.py.  The roundings counted there are
relative to a weight; what a kernel may lose of weights far below their neighbours' is not
counted, so the cases hold it to a share of the result that the tolerances leave open.
"""
import functools
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_07_b200 import synth, tqkv
from test_cross import CODECS, DEV, Call, Codec, U

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=None)
def codec_of(name, H):
    return Codec(*CODECS[name], H=H)


class Made(Call):
    """Every sequence's states around one logit: key t of a sequence gives about -below bits, or
    0 where it is a zero state (key and value); values of the given norms."""

    def __init__(self, cd, qlens, kvlens, G, zero, below, norms, seed=0):
        super().__init__(cd, qlens, kvlens, G, seed=seed)
        d, H, g = cd.d, cd.H, torch.Generator().manual_seed(seed + 10)
        u = torch.randn(d, generator=g, dtype=torch.float64)
        u /= u.norm()
        for slots in self.slots:
            n = len(slots)
            K = 0.3 * torch.randn((n, H, d), generator=g, dtype=torch.float64) - below * math.log(2) * u
            V = torch.randn((n, H, d), generator=g, dtype=torch.float64)
            V *= (torch.as_tensor(norms(np.arange(n)), dtype=torch.float64)[:, None, None] / V.norm(dim=2, keepdim=True))
            z = torch.as_tensor(zero(np.arange(n), n))
            K[z], V[z] = 0, 0
            tqkv.encode(cd.kp, cd.vp, cd.desc, *(x.to(torch.bfloat16).to(DEV).contiguous() for x in (K, V)),
                        torch.from_numpy(slots).to(DEV), self.cache)
        noise = torch.randn(self.Q.shape, generator=g, dtype=torch.float64)
        self.Q.copy_(math.sqrt(d) * u + 0.3 * noise)
        # A logit of size l is a sum of products that go as u_i^2, each off by two fp16 roundings (rms
        # 2^-11 / sqrt 3 of it at most), so by l 2^-11 sqrt(2/3 sum u_i^4), and the query's half of that
        # is the same for every key of a row: it does not average out in the 2-norm (1.2 times that here).
        self.share = below * math.log(2) * U * math.sqrt(float((u ** 4).sum()))

    def check_far(self, out, lse):
        """check where logits are large: 2^-8 and the share above for the 2-norm."""
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        err2 = ref2 = 0.0
        for pick, hs, ref, rl, tol, tl in self.reference():
            e, f = np.abs(o[pick, hs].reshape(ref.shape) - ref), np.abs(l[pick, hs].reshape(-1) - rl)
            assert (e <= tol).all() and (f <= tl).all(), ((e / tol).max(), (f / tl).max())
            err2, ref2 = err2 + (e ** 2).sum(), ref2 + (ref ** 2).sum()
        assert err2 <= (2.0 ** -8 + self.share) ** 2 * ref2, math.sqrt(err2 / ref2)


def constant(norm):
    return lambda t: np.full(len(t), norm)


ZEROS = {
    "start": lambda t, n: t < 128, "two tiles": lambda t, n: t < 256, "middle": lambda t, n: (t >= 256) & (t < 512),
    "end": lambda t, n: t >= n // 128 * 128 - 128,
}


@pytest.mark.parametrize("codec,qlens", [("k5v4", [70]), ("k5v4", [1]), ("d64", [70]), ("d64", [1])])
@pytest.mark.parametrize("length", [880, 1024])                       # seven tiles in one piece, eight in two
@pytest.mark.parametrize("where", list(ZEROS))
def test_zero_tiles(codec, qlens, length, where):
    for norm in (11.0, 0.1, 0.003):
        for below in (0, 4, 8):
            c = Made(codec_of(codec, 1), qlens, [length], 4, ZEROS[where], below, constant(norm))
            out, lse, flags = c.run()
            assert flags == 0
            c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64"])
@pytest.mark.parametrize("length", [700, 4096])
@pytest.mark.parametrize("below", [16, 30, 45])
def test_zero_tiles_far_above_the_rest(codec, length, below):
    """Tiles of zero states hold all of the sum and none of the result."""
    for where in ("start", "middle"):
        c = Made(codec_of(codec, 1), [70, 7], [length, 640], 2, ZEROS[where], below, constant(0.02))
        out, lse, flags = c.run()
        assert flags == 0
        c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64"])
def test_nothing_but_zero_states(codec):
    for qlens in ([70, 3], [1, 1]):
        c = Made(codec_of(codec, 2), qlens, [1024, 77], 2, lambda t, n: t >= 0, 0, constant(1.0))
        out, lse, flags = c.run()
        assert flags == 0 and (out[:sum(qlens)] == 0).all()
        c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64"])
@pytest.mark.parametrize("at", [0, 2000])
@pytest.mark.parametrize("below", [16, 20, 22, 24])
def test_one_strong_key_without_a_value(codec, at, below):
    """The result is made of weights below 2^-below of the largest alone."""
    for length in (880, 4096):
        c = Made(codec_of(codec, 1), [70], [length], 4, lambda t, n: t == at % n, below, constant(1.0))
        out, lse, flags = c.run()
        assert flags == 0
        c.check(out, lse)


@pytest.mark.parametrize("codec,qlens", [("k5v4", [70]), ("k5v4", [2]), ("d64", [70]), ("d64k8", [90])])
@pytest.mark.parametrize("length", [880, 4096])
def test_value_norms_that_differ_between_tiles(codec, qlens, length):
    steps = np.array([0, -8, 8, 3, -12, 6, -3])
    c = Made(codec_of(codec, 1), qlens, [length], 4, lambda t, n: t < 0, 0, lambda t: 2.0 ** steps[t // 128 % 7])
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64"])
@pytest.mark.parametrize("length", [880, 4096])
def test_loud_values_that_nothing_looks_at(codec, length):
    """Every other tile ends with a value 2^12 times the others' size whose weight is nothing."""
    cd = codec_of(codec, 1)
    c = Made(cd, [70], [length], 2, lambda t, n: t < 0, 0, lambda t: np.where(t % 256 == 127, 40.0, 0.01))
    loud = torch.from_numpy(c.slots[0][127::256].copy()).to(DEV)
    q = c.Q.double().mean((0, 1))
    K = (q / q.norm() * -40.0).to(torch.bfloat16).expand(len(loud), 1, cd.d).contiguous()
    V = synth.normal((len(loud), 1, cd.d), seed=77, device=DEV) * 4.0
    tqkv.encode(cd.kp, cd.vp, cd.desc, K, V, loud, c.cache)
    out, lse, flags = c.run()
    assert flags == 0
    c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64"])
@pytest.mark.parametrize("qlens", [[3, 1], [70, 9]])
def test_tiny_queries(codec, qlens):
    """Coordinates down to bf16's smallest: the mean of the values, and no other row changes."""
    c = Call(codec_of(codec, 2), qlens, [1100, 300], 2)
    ref, rl, _ = c.run()
    n = sum(qlens)
    tiny = {(0, 0): 2.0 ** -116, (0, 1): 1e-37, (1, 3): 2.0 ** -133, (n - 1, 2): 1e-36, (n - 1, 0): 0.0}
    keep = torch.ones(c.Q.shape[:2], dtype=torch.bool, device=DEV)
    for (row, head), x in tiny.items():
        c.Q[row, head] = (torch.randn(c.cd.d, generator=torch.Generator().manual_seed(row)).sign() * x).to(torch.bfloat16).to(DEV)
        keep[row, head] = False
    c.Q[0, 1, 5:] = 0                                                 # few coordinates that are not zero
    out, lse, flags = c.run()
    assert flags == 0 and torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], rl[keep])
    c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64", "d32"])
def test_no_queries_and_no_sequences(codec):
    """A step in which nothing is to be read: the call returns, and writes nothing."""
    c = Call(codec_of(codec, 2), [3, 0], [70, 9], 2)
    kp, vp, desc, Q, cu, max_q, table, lens, most, cache = c.args
    assert tqkv.cross_attn(kp, vp, desc, Q[:0], torch.zeros_like(cu), 0, table, lens, most, cache).shape == (0, *Q.shape[1:])
    assert tqkv.cross_attn(kp, vp, desc, Q[:0], torch.zeros_like(cu), max_q, table, lens, most, cache).numel() == 0
    assert (tqkv.cross_attn(kp, vp, desc, Q, cu[:1], max_q, table[:0], lens[:0], most, cache) == 0).all()
    assert (tqkv.cross_attn(kp, vp, desc, Q, torch.zeros_like(cu), max_q, table, lens, most, cache) == 0).all()


def test_rounds_of_long_table_rows():
    """Room for 440,000 states in pages of 8: table rows of 220 KB, so some 600 queries a round by
    rows; the last round has fewer rows and splits their keys."""
    for total in (1150, 1200):
        c = Call(Codec(*CODECS["d32"], P=8, H=1), [total - 5, 5], [300, 64], 1, extra_rows=3)
        wide = torch.full((2, 55_000), -1, dtype=torch.int32, device=DEV)
        wide[:, :c.table.shape[1]] = c.table
        c.maxkv = 440_000
        c.args = c.args[:6] + (wide, c.lens, c.maxkv, c.cache)
        out, lse, flags = c.run()
        assert flags == 0
        c.check(out, lse, rows=[0, 1, 4, 590, 605, 606, 607, 608, 609, 610, 611, 612, total - 6])


@pytest.mark.parametrize("codec", ["k5v4", "d64", "33"])
@pytest.mark.parametrize("length", [70, 130, 1500, 4096])
@pytest.mark.parametrize("below", [30, 60, 75])
def test_strong_keys_without_a_value_far_above(codec, length, below):
    """Their neighbours' weights alone make the result: keys 7, 707, 1407 and so on have no value."""
    for norm in (11.0, 0.003):
        c = Made(codec_of(codec, 1), [70, 7], [length, 70], 4, lambda t, n: t % 700 == 7, below, constant(norm))
        out, lse, flags = c.run()
        assert flags == 0
        c.check_far(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "k3v4", "k8v4", "frac", "polar", "33", "d32"])
@pytest.mark.parametrize("G", [4, 7])
def test_strong_keys_without_a_value_by_rows(codec, G):
    """Runs of a few queries: weights far below a key that has none of the result, values of any size."""
    cd = codec_of(codec, 1)
    for below, norm, length in ((16, 0.003, 1500), (20, 11.0, 1500), (24, 1.0, 4096), (30, 0.02, 130), (60, 1.0, 1500)):
        c = Made(cd, [2, 1], [length, 70], G, lambda t, n: t % 700 == 7, below, constant(norm))
        out, lse, flags = c.run()
        assert flags == 0
        c.check_far(out, lse)


def test_strong_keys_without_a_value_under_the_dense_rotation():
    cd = Codec(128, 4, True, 4, H=1, dense=True)
    for qlens in ([2, 1], [20, 9]):
        c = Made(cd, qlens, [1500, 70], 4, lambda t, n: t % 700 == 7, 24, constant(0.01))
        out, lse, flags = c.run()
        assert flags == 0
        c.check_far(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "k3v4", "d64", "d32"])
@pytest.mark.parametrize("norm", [2.0 ** -13, 4000.0])
def test_small_and_large_values(codec, norm):
    for qlens in ([2, 3], [70, 9]):
        c = Made(codec_of(codec, 2), qlens, [900, 64], 2, lambda t, n: t < 0, 0, constant(norm))
        out, lse, flags = c.run()
        assert flags == 0
        c.check(out, lse)


@pytest.mark.parametrize("codec", ["k5v4", "d64", "d32"])
@pytest.mark.parametrize("qlens", [[2, 1], [70, 9]])
def test_weights_at_the_end_of_the_stated_range(codec, qlens):
    """Keys without a value 2^64 above the others, whose values are small, and change size from tile to tile."""
    steps = np.array([-13, -9, -3, -13])
    for length in (1024, 3000):
        c = Made(codec_of(codec, 1), qlens, [length, 70], 2, lambda t, n: t % 300 == 7, 64, lambda t: 2.0 ** steps[t // 128 % 4])
        out, lse, flags = c.run()
        assert flags == 0
        c.check_far(out, lse)
