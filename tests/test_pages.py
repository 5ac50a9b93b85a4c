"""tq_pages_reserve / fork / compact / free against a sequential model of the block table.

Everything here is whole numbers and bytes, so every comparison is for equality: the tables,
lengths, reference counts, slots and every byte of every layer's cache after every call, and
the status word.
"""
import ctypes
import random

import numpy as np
import pytest
import torch

from kv_cache_vector_07_b200 import tqkv
from oracle import oracle as O

DEV = "cuda"


class Model:
    """The block table and the caches' bytes, one request after another."""

    def __init__(self, lay, P, H, num_blocks, n_rows, max_blocks, layers, seed=0):
        self.P, self.H, self.fields = P, H, list(lay.fields.values())
        r = np.random.default_rng(seed)
        self.caches = r.integers(0, 256, (layers, num_blocks, H, lay.page_bytes), dtype=np.uint8)
        self.refs = np.zeros(num_blocks, np.int32)
        self.table = r.integers(-5, num_blocks + 5, (n_rows, max_blocks), dtype=np.int32)
        self.lens = np.zeros(n_rows, np.int32)
        self.rows, self.width = n_rows, max_blocks

    def pages(self, n):
        return -(-int(n) // self.P)

    def _deal(self, needs):
        """Ranges of the lowest free pages for every request, None where they run out."""
        free, at, got = np.flatnonzero(self.refs == 0), 0, []
        for n in needs:
            got.append([] if n == 0 else None if n is None or at + n > len(free) else list(free[at:at + n]))
            at += n or 0
        return got

    def _live(self, ids):
        return all(0 <= i < len(self.refs) and self.refs[i] > 0 for i in ids)

    def reserve(self, new, n_slots):
        slots = np.full(n_slots, -1, np.int32)
        flags, needs, at, where = 0, [], 0, []
        for r in range(self.rows):
            add, n = max(int(new[r]), 0), int(self.lens[r])
            where.append(at)
            bad = 0
            if add and (n < 0 or at + add > n_slots):
                bad = tqkv.TQ_DEV_ROW
            elif add and self.pages(n + add) > self.width:
                bad = tqkv.TQ_DEV_NO_PAGES
            elif add and n % self.P:
                last = self.table[r, self.pages(n) - 1]
                if not self._live([last]):
                    bad = tqkv.TQ_DEV_BLOCK_RANGE
                elif self.refs[last] != 1:
                    bad = tqkv.TQ_DEV_PAGE_SHARED
            flags |= bad
            needs.append(None if bad or not add else self.pages(n + add) - self.pages(n))
            at += add
        for r, ids in enumerate(self._deal(needs)):
            add, n = max(int(new[r]), 0), int(self.lens[r])
            if needs[r] is None:
                continue
            if ids is None:
                flags |= tqkv.TQ_DEV_NO_PAGES
                continue
            self.table[r, self.pages(n):self.pages(n + add)] = ids
            self.refs[ids] = 1
            for t in range(add):
                pos = n + t
                slots[where[r] + t] = self.table[r, pos // self.P] * self.P + pos % self.P
            self.lens[r] += add
        return slots, flags

    def fork(self, src, dst):
        flags, needs, lens = 0, [], []
        for i, (s, d) in enumerate(zip(src, dst)):
            n = 0
            if not (0 <= s < self.rows and 0 <= d < self.rows) or list(dst).index(d) != i or self.lens[d] != 0 or \
                    not 0 <= self.lens[s] <= self.width * self.P:
                flags |= tqkv.TQ_DEV_ROW
                needs.append(None)
            elif not self._live(self.table[s, :self.pages(self.lens[s])]):
                flags |= tqkv.TQ_DEV_BLOCK_RANGE
                needs.append(None)
            else:
                n = int(self.lens[s])
                needs.append(int(n % self.P != 0))
            lens.append(n)
        for i, ids in enumerate(self._deal(needs)):
            if needs[i] is None:
                continue
            if ids is None:
                flags |= tqkv.TQ_DEV_NO_PAGES
                continue
            s, d, n = src[i], dst[i], lens[i]
            full = n // self.P
            self.table[d, :full] = self.table[s, :full]
            np.add.at(self.refs, self.table[s, :full], 1)
            if ids:
                self.caches[:, ids[0]] = self.caches[:, self.table[s, full]]
                self.table[d, full] = ids[0]
                self.refs[ids[0]] = 1
            self.lens[d] = n
        return flags

    def compact(self, rows, keep, kept):
        flags, needs, stay, before = 0, [], [], self.refs.copy()
        for i, r in enumerate(rows):
            n, k = (int(self.lens[r]) if 0 <= r < self.rows else 0), int(kept[i])
            bad = 0
            st = []
            if not 0 <= r < self.rows or list(rows).index(r) != i or not 0 <= n <= self.width * self.P:
                bad = tqkv.TQ_DEV_ROW
            elif not 0 <= k <= keep.shape[1]:
                bad = tqkv.TQ_DEV_KEEP_RANGE
            elif self.pages(k) > self.width:
                bad = tqkv.TQ_DEV_NO_PAGES
            elif not self._live(self.table[r, :self.pages(n)]):
                bad = tqkv.TQ_DEV_BLOCK_RANGE
            elif any(not 0 <= t < n for t in keep[i, :k]):
                bad = tqkv.TQ_DEV_KEEP_RANGE
            else:
                for j in range(self.pages(k)):
                    p = range(j * self.P, min(k, (j + 1) * self.P))
                    st.append(all(keep[i, q] == q for q in p) and
                              (len(p) == self.P or before[self.table[r, j]] == 1))
            flags |= bad
            needs.append(None if bad else sum(not s for s in st))
            stay.append(st)
        for i, ids in enumerate(self._deal(needs)):
            if needs[i] is None:
                continue
            if ids is None:
                flags |= tqkv.TQ_DEV_NO_PAGES
                continue
            r, k = rows[i], int(kept[i])
            old, n = self.table[r].copy(), int(self.lens[r])
            for j in range(max(self.pages(n), self.pages(k))):
                stays = j < self.pages(k) and stay[i][j]
                if j < self.pages(n) and not stays:
                    self.refs[old[j]] -= 1
                if j < self.pages(k) and not stays:
                    self.table[r, j] = to = ids.pop(0)
                    self.refs[to] = 1
                    for p in range(j * self.P, min(k, (j + 1) * self.P)):
                        t = int(keep[i, p])
                        for off, bpt in self.fields:
                            a, b = off + p % self.P * bpt, off + t % self.P * bpt
                            self.caches[:, to, :, a:a + bpt] = self.caches[:, old[t // self.P], :, b:b + bpt]
            self.lens[r] = k
        return flags

    def free(self, rows):
        flags = 0
        for r in rows:
            if not 0 <= r < self.rows or not 0 <= self.lens[r] <= self.width * self.P:
                flags |= tqkv.TQ_DEV_ROW
                if 0 <= r < self.rows:
                    self.lens[r] = 0
                continue
            for i in self.table[r, :self.pages(self.lens[r])]:
                if not self._live([i]):
                    flags |= tqkv.TQ_DEV_BLOCK_RANGE
                else:
                    self.refs[i] -= 1
            self.lens[r] = 0
        return flags


class Pair:
    """The model and the library's state beside it."""

    def __init__(self, d=64, kbits=2, qjl=True, vbits=4, P=16, H=2, num_blocks=40, n_rows=8, max_blocks=9, layers=2,
                 seed=0):
        lib = lambda b: tqkv.TQ_BITS_POLAR if b == "polar" else (tqkv.half_bits(b) if b != int(b) else int(b))
        self.desc = tqkv.cache_desc(d, lib(kbits), qjl, lib(vbits), page_tokens=P, n_kv_heads=H)
        self.m = Model(O.Layout(d, kbits, qjl, vbits, page_tokens=P), P, H, num_blocks, n_rows, max_blocks, layers, seed)
        self.load()

    def load(self):
        m = self.m
        self.caches = [torch.from_numpy(c).to(DEV) for c in m.caches]
        self.refs, self.table, self.lens = (torch.from_numpy(x).to(DEV) for x in (m.refs, m.table, m.lens))
        self.state = (self.refs, self.table, self.lens)
        self.ws = torch.zeros(tqkv.pages_workspace_bytes(len(m.refs), m.rows, m.width), dtype=torch.uint8, device=DEV)

    def load_state(self):
        """The model's tables into the tensors that are there."""
        for t, x in zip(self.state, (self.m.refs, self.m.table, self.m.lens)):
            t.copy_(torch.from_numpy(x))

    def ints(self, x):
        return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)

    def same(self, flags, what=""):
        m = self.m
        assert tqkv.read_status(self.ws) == flags, what
        assert np.array_equal(self.lens.cpu().numpy(), m.lens), what
        assert np.array_equal(self.table.cpu().numpy(), m.table), what
        assert np.array_equal(self.refs.cpu().numpy(), m.refs), what
        for a, b in zip(self.caches, m.caches):
            assert np.array_equal(a.cpu().numpy(), b), what

    def reserve(self, new, n_slots=None):
        n_slots = sum(max(int(x), 0) for x in new) if n_slots is None else n_slots
        got = torch.full((n_slots,), 77, dtype=torch.int32, device=DEV)
        tqkv.pages_reserve(self.desc, *self.state, self.ints(new), got, workspace=self.ws)
        slots, flags = self.m.reserve(new, n_slots)
        self.same(flags, ("reserve", new))
        assert np.array_equal(got.cpu().numpy(), slots)
        return flags

    def fork(self, src, dst):
        tqkv.pages_fork(self.desc, self.caches, *self.state, self.ints(src), self.ints(dst), workspace=self.ws)
        flags = self.m.fork(src, dst)
        self.same(flags, ("fork", src, dst))
        return flags

    def compact(self, rows, lists, kept=None):
        most = max([len(x) for x in lists] + [0])
        keep = np.full((len(lists), most), -9, np.int32)
        for i, x in enumerate(lists):
            keep[i, :len(x)] = x
        kept = [len(x) for x in lists] if kept is None else kept
        tqkv.pages_compact(self.desc, self.caches, *self.state, self.ints(rows), self.ints(keep).view(len(lists), most),
                           self.ints(kept), workspace=self.ws)
        flags = self.m.compact(rows, keep, kept)
        self.same(flags, ("compact", rows, kept))
        return flags

    def free(self, rows):
        tqkv.pages_free(self.desc, *self.state, self.ints(rows), workspace=self.ws)
        flags = self.m.free(rows)
        self.same(flags, ("free", rows))
        return flags


CODECS = [dict(), dict(d=128, kbits=4, P=64, H=1, num_blocks=17), dict(kbits=8, qjl=False, P=8, max_blocks=20, num_blocks=90),
          dict(kbits=3, vbits=3, H=3, layers=1), dict(d=16, kbits=2.5, vbits=3.5, P=32), dict(d=8, kbits=1, vbits=1, P=24),
          dict(d=32, kbits="polar", vbits="polar", H=1), dict(d=128, kbits=4, vbits=0, H=1, layers=3),
          dict(d=256, kbits=1, qjl=False, vbits=2, num_blocks=1500, n_rows=70, max_blocks=30, layers=1)]


@pytest.mark.gpu
@pytest.mark.parametrize("seed,kw", list(enumerate(CODECS)))
def test_random_life_of_a_pool(seed, kw):
    p = Pair(seed=seed, **kw)
    m, r = p.m, random.Random(seed)
    hit = 0
    for _ in range(60):
        op = r.choice(["reserve", "reserve", "fork", "compact", "free"])
        some = r.sample(range(m.rows), r.randint(1, m.rows))
        if op == "reserve":
            new = [r.choice([0, 0, 1, 1, m.P, r.randint(-2, 3 * m.P)]) for _ in range(m.rows)]
            n = sum(max(x, 0) for x in new)
            hit |= p.reserve(new, n + r.choice([0, 0, 0, 5, -min(n, 3)]))
        elif op == "fork":
            dst = r.sample(range(m.rows), r.randint(1, m.rows))
            hit |= p.fork([r.choice(some) for _ in dst], dst)
        elif op == "compact":
            lists = []
            for row in some:
                n = int(m.lens[row])
                keep = sorted(r.sample(range(n), r.randint(0, n)))
                how = r.random()
                if how < 0.25:
                    keep = list(range(r.randint(0, n)))                      # the last tokens dropped
                elif how < 0.4:
                    r.shuffle(keep)
                elif how < 0.5 and n:
                    keep = [r.randrange(n) for _ in range(r.randint(0, n + 5))]   # tokens named again
                lists.append(keep)
            hit |= p.compact(some, lists)
        else:
            hit |= p.free(some[:max(1, len(some) // 3)])
    assert hit & (tqkv.TQ_DEV_NO_PAGES | tqkv.TQ_DEV_ROW)            # the run met full pools or refused rows
    p.free(list(range(m.rows)))
    assert (m.refs == 0).all() and (m.lens == 0).all()


@pytest.mark.gpu
def test_requests_that_cannot_be_served():
    p = Pair(num_blocks=12, n_rows=6, max_blocks=4)
    P = p.m.P
    assert p.reserve([20, 2 * P, 0, 0, 0, 0]) == 0
    # rows out of range, a target in use, a target named twice, a row that forks itself
    assert p.fork([0, 0, 0, 9, 0, 1], [2, 2, 1, 3, -1, 1]) == tqkv.TQ_DEV_ROW
    assert p.fork([3], [3]) == 0 and p.fork([3], [4]) == 0                # an empty row copied
    # a chain in one call: row 3 is empty when row 4 takes it
    assert p.fork([1, 3], [3, 4]) == 0
    assert p.m.lens[3] == 2 * P and p.m.lens[4] == 0
    # the table row is too short, then the pool is
    assert p.reserve([0, 3 * P, 0, 0, 0, 0]) == tqkv.TQ_DEV_NO_PAGES
    assert p.reserve([0, 0, 0, 0, 4 * P, 4 * P]) == tqkv.TQ_DEV_NO_PAGES  # five pages in use, twelve in all
    assert p.m.lens[4] == 4 * P and p.m.lens[5] == 0
    assert p.reserve([1, 1, 1, 1, 0, 0]) == 0
    assert p.reserve([0, 0, 0, 0, 0, 2 * P]) == tqkv.TQ_DEV_NO_PAGES
    assert p.reserve([0, 0, 0, 0, 0, P]) == 0
    # tokens into a page that two rows read: only by the caller's own hand
    q = Pair()
    q.reserve([5, 0, 0, 0, 0, 0, 0, 0])
    q.m.table[1, 0], q.m.lens[1] = q.m.table[0, 0], 5
    q.m.refs[q.m.table[0, 0]] = 2
    q.load()
    assert q.reserve([1, 1, 0, 0, 0, 0, 0, 0]) == tqkv.TQ_DEV_PAGE_SHARED
    # compaction: kept tokens out of range, lists longer than the array, rows twice
    assert q.compact([0], [[5]]) == tqkv.TQ_DEV_KEEP_RANGE
    assert q.compact([0], [[-1]]) == tqkv.TQ_DEV_KEEP_RANGE
    assert q.compact([0], [[0, 1]], kept=[3]) == tqkv.TQ_DEV_KEEP_RANGE
    assert q.compact([0], [[0, 1]], kept=[-1]) == tqkv.TQ_DEV_KEEP_RANGE
    assert q.compact([0, 0, 99], [[1, 0], [1], [0]]) == tqkv.TQ_DEV_ROW
    assert q.compact([0], [[]]) == 0 and q.m.lens[0] == 0
    # free: twice, out of range, empty
    assert q.free([1, 1, 2, 2]) == 0
    assert q.free([-1, 8]) == tqkv.TQ_DEV_ROW


@pytest.mark.gpu
def test_tables_that_are_broken_are_reported():
    for page in (-1, 40, 39):                                             # below, behind, free
        p = Pair()
        p.reserve([20, 20, 0, 0, 0, 0, 0, 0])
        p.m.table[0, 1] = page
        p.load()
        assert p.fork([0, 1], [2, 3]) == tqkv.TQ_DEV_BLOCK_RANGE
        assert p.compact([0, 1], [[0], [0]]) == tqkv.TQ_DEV_BLOCK_RANGE
        assert p.reserve([1, 0, 0, 0, 0, 0, 0, 0]) == tqkv.TQ_DEV_BLOCK_RANGE
        assert p.free([0, 1]) == tqkv.TQ_DEV_BLOCK_RANGE
    for n in (-1, 9 * 16 + 1):
        p = Pair()
        p.m.lens[0] = n
        p.load()
        assert p.fork([0], [1]) == tqkv.TQ_DEV_ROW
        assert p.compact([0], [[0]]) == tqkv.TQ_DEV_ROW
        assert p.free([0]) == tqkv.TQ_DEV_ROW


@pytest.mark.gpu
def test_workspace_it_makes_belongs_to_its_stream():
    p, q = Pair(), Pair()
    new, slots = p.ints([20, 33, 0, 1, 0, 0, 0, 5]), torch.zeros(59, dtype=torch.int32, device=DEV)
    tqkv.pages_reserve(p.desc, *p.state, new, slots)
    side, other = torch.cuda.Stream(), torch.zeros_like(slots)
    busy = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(40):                                                   # a cleared workspace would come behind these
        busy += 1
    ws = tqkv.pages_reserve(q.desc, *q.state, new, other, stream=side)
    side.synchronize()
    assert tqkv.read_status(ws, side) == 0
    torch.cuda.synchronize()
    assert torch.equal(slots, other) and all(torch.equal(a, b) for a, b in zip(p.state, q.state))


@pytest.mark.gpu
def test_many_layers_and_no_requests():
    p = Pair(d=8, kbits=1, vbits=1, P=8, H=1, layers=131, num_blocks=9, n_rows=3, max_blocks=3)
    assert p.reserve([13, 0, 0]) == 0
    assert p.fork([0, 0], [1, 2]) == 0
    assert p.compact([1], [[1, 3, 12]]) == 0
    assert p.fork([], []) == 0 and p.free([]) == 0 and p.compact([], []) == 0 and p.reserve([0, 0, 0]) == 0


@pytest.mark.gpu
def test_layers_that_are_slices_of_one_tensor():
    """Their caches lie on 16 bytes, not on 256."""
    p = Pair(d=64, kbits=2, vbits=4, P=16, H=1, num_blocks=13, n_rows=4, max_blocks=4, layers=3)
    whole = torch.from_numpy(p.m.caches).to(DEV)
    p.caches = list(whole.unbind(0))
    assert any(c.data_ptr() % 256 for c in p.caches)
    assert p.reserve([20, 5, 0, 0]) == 0 and p.fork([0, 1], [2, 3]) == 0
    assert p.compact([2, 3], [[1, 19, 3], [4]]) == 0 and p.free([0, 1, 2, 3]) == 0


@pytest.mark.gpu
def test_large_pool_is_searched_to_its_end():
    n = 200000
    p = Pair(d=8, kbits=1, vbits=0, P=8, H=1, layers=1, num_blocks=n, n_rows=3, max_blocks=5000)
    p.m.refs[:] = 1
    free = [0, 1, 1023, 1024, 4095, 4096, 99999, n - 2, n - 1]
    p.m.refs[free] = 0
    p.load()
    assert p.reserve([8 * 4, 8 * 4 + 1, 8]) == tqkv.TQ_DEV_NO_PAGES        # 4, 5 and 1 pages: nine are there
    assert list(p.m.table[1, :5]) == free[4:] and p.m.lens[2] == 0


@pytest.mark.gpu
def test_more_rows_and_requests_than_shared_memory_holds():
    """The plans keep 1,024 requests and 4,096 rows on the chip, others in the workspace."""
    p = Pair(d=8, kbits=1, vbits=0, P=8, H=1, layers=1, num_blocks=9000, n_rows=5000, max_blocks=3)
    r = random.Random(1)
    assert p.reserve([r.randint(0, 12) if i < 2500 else 0 for i in range(5000)]) == 0
    src = [r.randrange(2500) for _ in range(1500)]
    dst = r.sample(range(2490, 5000), 1500)                  # some of them in use
    assert p.fork(src, dst) == tqkv.TQ_DEV_ROW
    rows = r.sample(range(5000), 1300)
    lists = [sorted(r.sample(range(int(p.m.lens[x])), r.randint(0, int(p.m.lens[x])))) for x in rows]
    assert p.compact(rows, lists) == 0
    assert p.free(list(range(5000))) == 0
    assert (p.m.refs == 0).all()


@pytest.mark.gpu
def test_captured_calls_replay_on_the_state_they_find():
    p = Pair()
    p.reserve([20, 0, 0, 0, 0, 0, 0, 0])
    src, dst = p.ints([0, 0]), p.ints([1, 2])
    new, slots = p.ints([0, 3, 3, 0, 0, 0, 0, 0]), p.ints([0] * 6)
    keep, kept = p.ints([[0, 2, 19, 22], [1, 2, 3, 4]]), p.ints([4, 2])
    args = (p.desc, p.caches, *p.state)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tqkv.pages_fork(*args, src, dst, workspace=p.ws)
        tqkv.pages_reserve(p.desc, *p.state, new, slots, workspace=p.ws)
        tqkv.pages_compact(*args, dst, keep, kept, workspace=p.ws)
        tqkv.pages_free(p.desc, *p.state, dst, workspace=p.ws)
    for length in (20, 21, 32):
        p.m.reserve([length - int(p.m.lens[0])] + [0] * 7, 64)
        p.load_state()
        g.replay()
        torch.cuda.synchronize()
        flags = p.m.fork([0, 0], [1, 2])
        want, more = p.m.reserve([0, 3, 3, 0, 0, 0, 0, 0], 6)
        flags |= more | p.m.compact([1, 2], np.array([[0, 2, 19, 22], [1, 2, 3, 4]]), [4, 2]) | p.m.free([1, 2])
        p.same(flags, length)
        assert np.array_equal(slots.cpu().numpy(), want)


def _c(name, desc=None, pool=None, ws=256, ws_bytes=1 << 30, **kw):
    desc = tqkv.cache_desc(64, 2, True, 4, page_tokens=16, n_kv_heads=2) if desc is None else desc
    pool = dict(dict(refs=256, table=256, lens=256, num_blocks=10, n_rows=4, max_blocks=3), **(pool or {}))
    pool = tqkv._PagePool(*[pool[f] for f, _ in tqkv._PagePool._fields_])
    caches = (ctypes.c_void_p * 2)(*kw.pop("caches", (256, 512)))
    a = dict(n_layers=2, n=1, ints=256, n_slots=1, keep_stride=2, keep=256)
    a.update(kw)
    d, p = ctypes.byref(desc), ctypes.byref(pool)
    if name == "reserve":
        return tqkv._lib.tq_pages_reserve(d, p, a["ints"], a["ints"], a["n_slots"], ws, ws_bytes, None)
    if name == "fork":
        return tqkv._lib.tq_pages_fork(d, p, caches, a["n_layers"], a["ints"], a["ints"], a["n"], ws, ws_bytes, None)
    if name == "compact":
        return tqkv._lib.tq_pages_compact(d, p, caches, a["n_layers"], a["ints"], a["keep"], a["keep_stride"], a["ints"],
                                          a["n"], ws, ws_bytes, None)
    return tqkv._lib.tq_pages_free(d, p, a["ints"], a["n"], ws, ws_bytes, None)


@pytest.mark.parametrize("name", ["reserve", "fork", "compact", "free"])
@pytest.mark.parametrize("kw", [
    dict(desc=tqkv.cache_desc(100, 2, True, 4)), dict(ws=None), dict(ws=128), dict(ws_bytes=256), dict(ints=None),
    dict(ints=258), dict(pool=dict(refs=None)), dict(pool=dict(table=None)), dict(pool=dict(lens=None)),
    dict(pool=dict(lens=257)), dict(pool=dict(num_blocks=0)), dict(pool=dict(num_blocks=1 << 31)),
    dict(pool=dict(num_blocks=(1 << 31) // 16)), dict(pool=dict(n_rows=0)), dict(pool=dict(max_blocks=0)),
    dict(pool=dict(max_blocks=(1 << 31) // 16))])
def test_c_refusals(name, kw):
    assert _c(name, **kw) == tqkv.TQ_EINVAL


@pytest.mark.parametrize("name,kw", [
    ("reserve", dict(n_slots=-1)), ("fork", dict(n=-1)), ("fork", dict(n=5)), ("fork", dict(n_layers=0)),
    ("fork", dict(caches=(256, None))), ("fork", dict(caches=(256, 300))), ("compact", dict(n=5)),
    ("compact", dict(keep_stride=-1)), ("compact", dict(keep=None)), ("compact", dict(caches=(None, 256))),
    ("free", dict(n=-1))])
def test_c_refusals_of_single_arguments(name, kw):
    assert _c(name, **kw) == tqkv.TQ_EINVAL


def test_workspace_bytes():
    assert tqkv.pages_workspace_bytes(0, 1, 1) == tqkv.pages_workspace_bytes(1, 0, 1) == tqkv.pages_workspace_bytes(1, 1, 0) == 0
    assert tqkv.pages_workspace_bytes(1000, 8, 16) < tqkv.pages_workspace_bytes(100000, 8, 16)


def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        tqkv.pages_free(tqkv.cache_desc(64, 2, True, 4), i, i.view(2, 2), i[:2], i)


@pytest.mark.gpu
def test_binding_refusals():
    p = Pair()
    rows = p.ints([0])
    bad = [
        lambda: tqkv.pages_free(p.desc, p.refs.long(), p.table, p.lens, rows),
        lambda: tqkv.pages_free(p.desc, p.refs, p.table[:, :3], p.lens, rows),
        lambda: tqkv.pages_free(p.desc, p.refs, p.table, p.lens[:3], rows),
        lambda: tqkv.pages_free(p.desc, p.refs, p.table, p.lens, rows.view(1, 1)),
        lambda: tqkv.pages_fork(p.desc, [], *p.state, rows, rows),
        lambda: tqkv.pages_fork(p.desc, [p.caches[0][:5]], *p.state, rows, rows),
        lambda: tqkv.pages_fork(p.desc, p.caches, *p.state, rows, p.ints([0, 1])),
        lambda: tqkv.pages_compact(p.desc, p.caches, *p.state, rows, p.ints([0]), rows),
        lambda: tqkv.pages_compact(p.desc, p.caches, *p.state, rows, p.ints([[0], [1]]), rows),
        lambda: tqkv.pages_reserve(p.desc, *p.state, rows, rows),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    small = torch.zeros(512, dtype=torch.uint8, device=DEV)
    with pytest.raises(tqkv.TQError):
        tqkv.pages_free(p.desc, *p.state, rows, workspace=small)
