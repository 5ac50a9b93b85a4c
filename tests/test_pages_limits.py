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
