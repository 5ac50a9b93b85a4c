"""The pages calls at the ends of their arguments' ranges (refusals on the host: the pointers are made up)."""
import pytest

from kv_cache_vector_07_b200 import tqkv
from test_pages import _c

TOP = 2 ** 31


@pytest.mark.parametrize("name,kw", [
    ("free", dict(n=TOP - 1)), ("free", dict(n=TOP - 8)), ("free", dict(n=TOP - 1024)),
    *[(name, dict(pool=dict(n_rows=TOP - 1), ws_bytes=1 << 60)) for name in ("reserve", "fork", "compact", "free")],
    *[(name, dict(pool=dict(max_blocks=(TOP - 16) // 16), ws_bytes=1 << 60)) for name in ("reserve", "fork", "compact", "free")],
    *[(name, dict(pool=dict(num_blocks=(TOP - 16) // 16), ws_bytes=1 << 60)) for name in ("reserve", "fork", "compact", "free")]])
def test_counts_that_a_loop_would_step_past(name, kw):
    assert _c(name, **kw) == tqkv.TQ_EINVAL


BASE = dict(refs=1 << 12, table=2 << 12, lens=3 << 12, num_blocks=10, n_rows=4, max_blocks=3)      # 40, 48 and 16 bytes


def _calls(ints, ws=1 << 20, **pool):
    """The codes of the four calls, every request at `ints`."""
    kw = dict(pool=dict(BASE, **pool), ws=ws, ints=ints)
    return [_c("reserve", **dict(kw, n_slots=0)), _c("fork", **kw), _c("compact", **dict(kw, keep=5 << 12)), _c("free", **kw)]


@pytest.mark.parametrize("name", ["refs", "table", "lens"])
def test_requests_within_the_pool(name):
    size = dict(refs=40, table=48, lens=16)[name]
    assert _calls(BASE[name]) == _calls(BASE[name] + size - 4) == [tqkv.TQ_EINVAL] * 4


def test_arrays_that_overlap():
    assert _calls(1 << 20) == _calls((1 << 20) + 256) == [tqkv.TQ_EINVAL] * 4                      # the workspace
    assert _calls(4 << 12, ws=2 << 12) == [tqkv.TQ_EINVAL] * 4
    assert _calls(4 << 12, lens=BASE["table"] + 44) == _calls(4 << 12, refs=BASE["lens"] - 36) == [tqkv.TQ_EINVAL] * 4
    kw = dict(pool=BASE, ws=1 << 20, ints=4 << 12)
    assert _c("reserve", **dict(kw, n_slots=9)) == tqkv.TQ_EINVAL                                   # new_tokens and slot_mapping
    assert _c("compact", **dict(kw, keep=BASE["lens"] - 4, keep_stride=2)) == tqkv.TQ_EINVAL


@pytest.mark.gpu
def test_workspaces_that_are_not_what_they_count():
    """A repeated byte counts as many as a workspace; a step of two is longer than it counts."""
    import torch

    from test_pages import DEV, Pair

    p = Pair()
    rows, need = p.ints([0]), p.ws.numel()
    byte = torch.zeros(1, dtype=torch.uint8, device=DEV)
    for ws in (byte.expand(1 << 20), torch.zeros(2 * need, dtype=torch.uint8, device=DEV)[::2]):
        for call in (lambda: tqkv.pages_free(p.desc, *p.state, rows, workspace=ws),
                     lambda: tqkv.pages_fork(p.desc, p.caches, *p.state, rows, rows, workspace=ws),
                     lambda: tqkv.pages_reserve(p.desc, *p.state, torch.zeros_like(p.state[2]), p.ints([0, 0]), workspace=ws),
                     lambda: tqkv.pages_compact(p.desc, p.caches, *p.state, rows, p.ints([[0]]), rows, workspace=ws)):
            with pytest.raises(ValueError):
                call()
