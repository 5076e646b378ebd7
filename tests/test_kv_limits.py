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


@pytest.mark.parametrize("scale,code", [(2.358e38, ALIGN), (-2.358e38, ALIGN), (2.4e38, SHAPE), (-2.9e38, SHAPE),
                                        (3.4e38, SHAPE)])
def test_scales_whose_logarithm_to_base_two_is_infinite(lib, scale, code):  # noqa: F811
    """Refused; the others are refused only for the misaligned `out` that comes later."""
    assert lib.ssd_kv_attention(cache(), P, None, P, ST, 0, 2, 3, 8, scale, 0, 0, ctypes.c_void_p(4104), None, P, 1 << 30,
                                None) == code
