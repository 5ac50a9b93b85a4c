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
