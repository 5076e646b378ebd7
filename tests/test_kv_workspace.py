"""A workspace made for n_q query tokens serves every call of fewer (no GPU needed)."""
import ctypes

import pytest

from speculative_decoding_verification_draft_gb300 import ssdv
from test_kv_abi import P, ST, cache, lib  # noqa: F401

WORKSPACE = 9


@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("per", [1, 2, 3, 4, 5, 7, 8, 13, 16, 24, 64, 128])
def test_size_never_falls(lib, head_dim, per):  # noqa: F811
    sizes = [lib.ssd_kv_workspace_bytes(n, 2 * per, 2, head_dim) for n in range(33)]
    assert sizes == sorted(sizes) and sizes[0] == 256


@pytest.mark.parametrize("head_dim,n_q,per", [(128, 9, 4), (128, 9, 8), (64, 32, 4), (256, 5, 8)])
def test_fewer_queries_than_it_was_made_for(lib, head_dim, n_q, per):  # noqa: F811
    """The refusal of a misaligned `out` comes after the workspace's: it is what every smaller call is refused for."""
    size = lib.ssd_kv_workspace_bytes(n_q, 2 * per, 2, head_dim)
    for n in range(1, n_q + 1):
        for dtype in (0, 1):
            status = lib.ssd_kv_attention(cache(head_dim=head_dim), P, None, P, ST, dtype, 2, n, 2 * per, 0.1, 0, 0,
                                          ctypes.c_void_p(4104), None, P, size, None)
            assert ssdv.STATUS_NAMES[status] == "SSD_ERR_ALIGN", (n, dtype)


def test_capture_id_arguments(lib):  # noqa: F811
    assert ssdv.STATUS_NAMES[lib.ssd_stream_capture_id(None, None)] == "SSD_ERR_NULL"
