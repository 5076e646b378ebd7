"""Arguments at the ends of their ranges (no GPU needed)."""
import ctypes

import pytest

from test_kv_abi import P, ST, cache, lib  # noqa: F401

SHAPE, ALIGN = 2, 4


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 31, (1 << 31) - 1])
def test_more_tokens_than_positions(lib, n):  # noqa: F811
    c = cache(n_kv_heads=1, head_dim=64)
    assert lib.ssd_kv_append(c, P, P, P, ST, P, ST, 0, 1, n, P, 1 << 10, None) == SHAPE
    assert lib.ssd_kv_read(c, P, P, 0, 1, n, P, P, P, 1 << 10, None) == SHAPE
