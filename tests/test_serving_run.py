"""The calls of a serving loop together, as they would be used: head norms with positions ->
pages reserved -> tokens written -> rows forked -> decode steps -> tokens dropped -> attention
over another row's states -> pages freed, in two layers that share one block table; and one
step captured into a graph and replayed.

What every attention call returns is compared with the formula in 64 bits over the bytes that
the cache holds (tolerances: test_cross.Codec.attend, whose counts of roundings also cover the
decode kernels: they take fp32 or split fp16 operands and round once to bf16, on top of which
parity.py allows the decode path 2e-3 for its fp32 sums).
"""
import numpy as np
import pytest
import torch

from kv_cache_vector_07_b200 import tqkv
from test_cross import Codec

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Loop:
    """Six rows of a block table over two layers."""

    def __init__(self, d, kbits, P, H, G, seed=0):
        self.cd = Codec(d, kbits, kbits != 8, 4, P=P, H=H)
        self.d, self.P, self.H, self.Hq, self.rows, self.width, self.blocks = d, P, H, H * G, 6, 160 // P + 2, 80
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.caches = [tqkv.alloc_cache(self.cd.desc, self.blocks) for _ in range(2)]
        for c in self.caches:
            c.random_(0, 256)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.refs, self.table, self.lens = torch.zeros(self.blocks, **i32), torch.full((self.rows, self.width), -1, **i32), torch.zeros(self.rows, **i32)
        self.ws = torch.zeros(tqkv.pages_workspace_bytes(self.blocks, self.rows, self.width), dtype=torch.uint8, device=DEV)
        self.rope = tqkv.rope_desc(d)
        self.inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().to(DEV)
        self.w = [1 + 0.1 * torch.randn(d, generator=self.g, device=DEV) for _ in range(2)]

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def project(self, n):
        """Slices of a QKV projection of n tokens: normed, rotated q and k, and v."""
        qkv = torch.randn((n, self.Hq + 2 * self.H, self.d), generator=self.g, device=DEV).bfloat16()
        return qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.H], qkv[:, self.Hq + self.H:].contiguous()

    def reserve(self, new, slots):
        tqkv.pages_reserve(self.cd.desc, self.refs, self.table, self.lens, new, slots, workspace=self.ws)

    def slots_of(self, row, upto=None):
        table, n = self.table.cpu().numpy(), int(self.lens[row]) if upto is None else upto
        pos = np.arange(n)
        return (table[row, pos // self.P] * self.P + pos % self.P).astype(np.int32)

    def check(self, layer, Q, out, rows):
        """out [rows, Hq, d] of queries Q over the rows' tokens."""
        raw = self.caches[layer].view(-1, self.caches[layer].shape[-1]).cpu().numpy()
        Q, out = Q.double().cpu().numpy(), out.double().cpu().numpy()
        G = self.Hq // self.H
        for i, r in enumerate(rows):
            for h in range(self.H):
                hs = slice(h * G, (h + 1) * G)
                ref, _, tol, _ = self.cd.attend(Q[i, hs], *self.cd.states(raw, self.slots_of(r), h))
                assert (np.abs(out[i, hs] - ref) <= tol + 2e-3).all(), (layer, r, np.abs(out[i, hs] - ref).max())

    def step(self, layer, q, k, v, slots, out=None, ws=None):
        """One decode step of every row."""
        qn, kn = tqkv.qk_norm_rope(self.rope, q, k, (self.lens - 1).clamp(min=0), self.inv, *self.w)
        return qn, tqkv.decode_step(self.cd.kp, self.cd.vp, self.cd.desc, kn, v, slots, qn, self.table, self.lens,
                                    self.width * self.P, self.caches[layer], out=out, workspace=ws)


@pytest.mark.parametrize("d,kbits,P,H,G", [(64, 4, 16, 2, 2), (128, 2, 64, 2, 4), (128, 8, 64, 1, 2)])
def test_loop(d, kbits, P, H, G):
    s = Loop(d, kbits, P, H, G)
    prompt = [37, 70, 0, 0, 0, 0]
    n = sum(prompt)
    slots = s.ints([-7] * (n + 3))
    s.reserve(s.ints(prompt), slots)
    assert (slots[n:] == -1).all() and (slots[:n] >= 0).all()
    pos = s.ints(list(range(37)) + list(range(70)) + [0] * 3)
    for c in s.caches:
        q, k, v = s.project(n + 3)
        _, kn = tqkv.qk_norm_rope(s.rope, q, k, pos, s.inv, *s.w)
        tqkv.encode(s.cd.kp, s.cd.vp, s.cd.desc, kn, v, slots, c)    # the last three have no slot
    tqkv.pages_fork(s.cd.desc, s.caches, s.refs, s.table, s.lens, s.ints([0, 0, 1]), s.ints([2, 3, 4]), workspace=s.ws)
    assert s.lens.tolist() == [37, 70, 37, 37, 70, 0]
    # two decode steps: every row goes its own way, the shared pages stay as they are
    shared = s.slots_of(0, 37 // P * P)
    before = [c.view(-1, c.shape[-1]).clone() for c in s.caches]
    for _ in range(2):
        slots = s.ints([0] * 5)
        s.reserve(s.ints([1, 1, 1, 1, 1, 0]), slots)
        slots = torch.cat([slots, s.ints([-1])])
        for layer in range(2):
            q, k, v = s.project(s.rows)
            qn, out = s.step(layer, q, k, v, slots)
            s.check(layer, qn, out, range(6))
            assert (out[5] == 0).all()
    for layer, c in enumerate(s.caches):
        for page in np.unique(shared // P):
            rows = slice(page * H, (page + 1) * H)
            assert torch.equal(c.view(-1, c.shape[-1])[rows], before[layer][rows])
    # rejected tokens, and a window with the first four kept
    keep = [list(range(36)), [0, 1, 2, 3] + list(range(20, 72))]
    lists = torch.zeros((2, 56), dtype=torch.int32, device=DEV)
    for i, x in enumerate(keep):
        lists[i, :len(x)] = s.ints(x)
    was = [s.slots_of(2), s.slots_of(4)]
    raw = [c.clone() for c in s.caches]
    tqkv.pages_compact(s.cd.desc, s.caches, s.refs, s.table, s.lens, s.ints([2, 4]), lists, s.ints([36, 56]), workspace=s.ws)
    assert s.lens.tolist() == [39, 72, 36, 39, 56, 0]
    for layer, c in enumerate(s.caches):
        for i, r in enumerate((2, 4)):
            for h in range(H):
                now = s.cd.states(c.view(-1, c.shape[-1]).cpu().numpy(), s.slots_of(r), h)
                then = s.cd.states(raw[layer].view(-1, c.shape[-1]).cpu().numpy(), was[i][keep[i]], h)
                assert all(np.array_equal(a, b) for a, b in zip(now, then))
        q, _, _ = s.project(s.rows)
        q = q.contiguous()
        out = tqkv.decode_attn(s.cd.kp, s.cd.vp, s.cd.desc, q, s.table, s.lens, s.width * s.P, c)
        s.check(layer, q, out, range(6))
        # runs of queries over the same rows, as an encoder's states
        runs = [3, 20, 0, 1, 40, 2]
        q, _, _ = s.project(sum(runs))
        q = q.contiguous()
        cu = s.ints([0] + list(np.cumsum(runs)))
        out = tqkv.cross_attn(s.cd.kp, s.cd.vp, s.cd.desc, q, cu, 40, s.table, s.lens, s.width * s.P, c)
        s.check(layer, q, out, [r for r, m in enumerate(runs) for _ in range(m)])
    assert tqkv.read_status(s.ws) == 0
    tqkv.pages_free(s.cd.desc, s.refs, s.table, s.lens, s.ints([0, 1, 2, 3, 4, 5]), workspace=s.ws)
    assert (s.refs == 0).all() and (s.lens == 0).all() and tqkv.read_status(s.ws) == 0


def test_captured_step_replays_as_the_eager_one():
    loops = [Loop(128, 2, 64, 2, 4, seed=5) for _ in range(2)]
    prompt = [60, 64, 7, 0, 0, 0]
    for s in loops:
        slots = s.ints([0] * 131)
        s.reserve(s.ints(prompt), slots)
        q, k, v = s.project(131)
        pos = s.ints(list(range(60)) + list(range(64)) + list(range(7)))
        _, kn = tqkv.qk_norm_rope(s.rope, q, k, pos, s.inv, *s.w)
        for c in s.caches:
            c.zero_()
            tqkv.encode(s.cd.kp, s.cd.vp, s.cd.desc, kn, v, slots, c)
    a, b = loops
    steps = [a.project(a.rows) for _ in range(8)]
    new, slots = b.ints([1, 1, 1, 0, 0, 0]), [x.ints([-1] * 6) for x in loops]
    buf = [t.clone() for t in steps[0]]
    out = torch.empty_like(buf[0].contiguous())
    ws = torch.zeros(tqkv.decode_workspace_bytes(b.cd.desc, b.rows, b.Hq, b.width * b.P), dtype=torch.uint8, device=DEV)
    saved = [t.clone() for t in (b.refs, b.table, b.lens, *b.caches)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                            # once outside the graph, then the state put back
        b.reserve(new, slots[1])
        b.step(0, *buf, slots[1], out=out, ws=ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.reserve(new, slots[1])
        b.step(0, *buf, slots[1], out=out, ws=ws)
    for t, x in zip((b.refs, b.table, b.lens, *b.caches), saved):
        t.copy_(x)
    for qkv in steps:                                        # the rows cross a page border on the way
        a.reserve(new, slots[0])
        _, want = a.step(0, *qkv, slots[0])
        for t, x in zip(buf, qkv):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:3], want[:3]) and torch.equal(slots[0], slots[1])
    for x, y in ((a.refs, b.refs), (a.table, b.table), (a.lens, b.lens), (a.caches[0], b.caches[0])):
        assert torch.equal(x, y)
