"""A request that visits a bad page: its queries' rows are NaN, the rows past its count what they always are."""
import numpy as np
import pytest
import torch

import kv_common as kc
from test_gpu_kv_attention import fill, ssdv  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n,G,D,dtype", [(5, 2, 128, BF16), (5, 5, 128, BF16), (5, 8, 128, BF16), (9, 8, 128, BF16),
                                         (5, 2, 64, F32), (5, 4, 256, BF16)])
def test_rows_past_the_count_of_a_bad_page(ssdv, n, G, D, dtype):  # noqa: F811
    """One short request, and one long enough to be split between CTAs, with bad pages in the middle."""
    lens, n_q = np.array([40, 9001, 33]), np.array([3, 2, n])
    p = kc.Pool(ssdv, 3, 1, D, 16, 9001 + n)
    fill(p, lens, lens + n_q)
    p.table[0, 1] = p.cache.shape[0]
    p.table[1, 300] = -1
    q, _ = kc.rows((3, n, G, D), dtype, 3)
    ws = ssdv.make_kv_workspace(n, G, 1, D)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, n_q=kc.ints(n_q), return_lse=True, workspace=ws)
    assert ssdv.read_status(ws) == 12
    for b in (0, 1):
        m = int(n_q[b])
        assert bool(torch.isnan(out[b, :m]).all()) and bool(torch.isnan(lse[b, :m]).all()), b
        assert bool((out[b, m:] == 0).all()) and bool((lse[b, m:] == -np.inf).all()), b
    assert bool(torch.isfinite(out[2]).all()) and bool(torch.isfinite(lse[2]).all())
