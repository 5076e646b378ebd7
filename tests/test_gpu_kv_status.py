"""What the status word of the cache calls' own workspaces tells."""
import pytest
import torch

import kv_common as kc
from test_gpu_kv_attention import ssdv  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
LENGTH = 13


@pytest.mark.parametrize("on_a_stream", [False, True])
def test_status_outlives_a_larger_workspace(ssdv, monkeypatch, on_a_stream):  # noqa: F811
    """An append's error is still told after an attention call that needs a larger workspace."""
    monkeypatch.setattr(ssdv, "_kv_ws_cache", {})
    stream = torch.cuda.Stream() if on_a_stream else None
    p = kc.Pool(ssdv, 2, 1, 128, 16, 64)
    k, _ = kc.rows((2, 5, 1, 128), BF16, 1)
    q, _ = kc.rows((2, 5, 8, 128), BF16, 2)
    bad, good = kc.ints([0, -1]), kc.ints([0, 0])
    torch.cuda.synchronize()
    ssdv.kv_append(p.cache, p.table, bad, k, k, stream=stream)
    small = ssdv.kv_workspace(stream=stream).numel()
    ssdv.kv_attention(p.cache, p.table, good, q, stream=stream)
    ws = ssdv.kv_workspace(stream=stream)
    assert ws.numel() > small
    assert ssdv.read_status(ws, stream=stream) == LENGTH
    ssdv.kv_attention(p.cache, p.table, good, q, stream=stream)
    assert ssdv.read_status(ws, stream=stream) == 0
