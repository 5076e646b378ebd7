"""Cache calls captured without a workspace: their status can be read, and captures share nothing."""
import numpy as np
import pytest
import torch

import kv_common as kc
from test_gpu_kv_attention import compare, ssdv  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def capture(ssdv, p, at, k, q, out=None):  # noqa: F811
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssdv.kv_append(p.cache, p.table, at, k, k)
        out, lse = ssdv.kv_attention(p.cache, p.table, at, q, return_lse=True)
        ws = ssdv.kv_workspace()
    return graph, ws, out, lse


def test_status_of_captured_calls(ssdv):  # noqa: F811
    """kv_workspace, asked inside the capture, gives the workspace whose status word the replays set."""
    p = kc.Pool(ssdv, 2, 1, 128, 16, 64)
    k, k64 = kc.rows((2, 5, 1, 128), BF16, 1)
    q, q64 = kc.rows((2, 5, 8, 128), BF16, 2)
    at = kc.ints([0, 0])
    eager = ssdv.kv_workspace()
    graph, ws, out, lse = capture(ssdv, p, at, k, q)
    assert ws is not None and ws is not eager
    at.copy_(kc.ints([0, -1]))
    graph.replay()
    assert ssdv.read_status(ws) == 13
    at.copy_(kc.ints([0, 30]))
    graph.replay()
    at.copy_(kc.ints([0, 0]))
    graph.replay()
    assert ssdv.read_status(ws) == 0
    compare(p, q, q64, kc.held(k64), kc.held(k64), np.zeros(2, int), np.full(2, 5), BF16, out, lse)
    assert ssdv.kv_workspace() is eager


def test_captures_and_eager_calls_do_not_share(ssdv):  # noqa: F811
    """A later capture on the same stream has its own workspace, and one graph's error is not told by the other."""
    p = kc.Pool(ssdv, 2, 1, 128, 16, 64)
    k, _ = kc.rows((2, 5, 1, 128), BF16, 1)
    q, _ = kc.rows((2, 5, 8, 128), BF16, 2)
    at, bt = kc.ints([0, 0]), kc.ints([0, 0])
    one, ws1, *_ = capture(ssdv, p, at, k, q)
    two, ws2, *_ = capture(ssdv, p, bt, k, q)
    assert ws1.data_ptr() != ws2.data_ptr()
    at.copy_(kc.ints([-1, 0]))
    one.replay()
    two.replay()
    assert ssdv.read_status(ws1) == 13 and ssdv.read_status(ws2) == 0
