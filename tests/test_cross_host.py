"""Sizes and refusals of tq_cross_attn that need no GPU."""
import pytest

from kv_cache_vector_07_b200 import tqkv

DESCS = [(128, 2, 64), (128, 4, 16), (64, 4, 64), (32, 4, 8), (256, 4, 64)]


def _desc(d, bits, P, H=2):
    return tqkv.cache_desc(d, bits, True, 4, page_tokens=P, n_kv_heads=H)


@pytest.mark.parametrize("d,bits,P", DESCS)
def test_workspace_of_nothing(d, bits, P):
    """No queries, no sequences, no room for a token: a size, and the calls do nothing."""
    for B, total, most, kv in ((2, 0, 4, 64), (2, 0, 0, 64), (0, 0, 0, 0), (0, 8, 4, 64), (2, 8, 0, 64), (2, 8, 4, 0)):
        assert 0 < tqkv.cross_workspace_bytes(_desc(d, bits, P), B, total, most, 4, kv) < 1 << 20
    assert tqkv.decode_workspace_bytes(_desc(d, bits, P), 0, 4, 64) > 0


@pytest.mark.parametrize("d,P,Hq,kv", [(32, 8, 2, 1 << 20), (256, 8, 2, 1 << 17), (256, 64, 16, 1 << 10), (32, 8, 2, 1 << 10)])
def test_workspace_by_rows_does_not_grow_with_the_call(d, P, Hq, kv):
    """Head sizes that go by rows: 128 MB a round of queries (prepared queries, partial results,
    a table row each), and 2,400 x G partial results where a round's keys are split."""
    sizes = [tqkv.cross_workspace_bytes(_desc(d, 4, P), 4, n, n, Hq, kv) for n in (1, 100, 10_000, 1_000_000)]
    most = (1 << 27) + 2400 * (Hq // 2) * (d + 2) * 4 + 4096
    assert all(0 < x <= most for x in sizes), sizes


def test_workspace_of_long_states_is_the_tiles():
    """1 GB of operand tiles and what goes with them, not a table row for every query."""
    assert tqkv.cross_workspace_bytes(_desc(64, 4, 16, H=8), 4, 65536, 65536, 8, 1 << 20) < 1.1 * 2 ** 30


def test_one_query_of_very_long_states():
    """A round holds one query at least: its table row and what the decode kernels need."""
    n = tqkv.cross_workspace_bytes(_desc(32, 4, 8), 1, 50, 50, 2, 1 << 30)
    assert 4 << 27 <= n <= (4 << 27) + (1 << 21)
