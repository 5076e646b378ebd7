"""What the attention tests check at few rows a kv head, at numbers of rows for which bf16 heads of 128 take
tcgen05: 20 and 40 (one pass), 72 (two passes)."""
import numpy as np
import pytest
import torch

import kv_common as kc
from test_gpu_kv_attention import check, compare, fill, ssdv  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROWS = pytest.mark.parametrize("n,G", [(5, 4), (5, 8), (9, 8)])


@ROWS
def test_errors_stay_with_their_request(ssdv, n, G):  # noqa: F811
    """Bad lengths and pages, one of them in the middle of a request that is split between CTAs."""
    B, Hkv, D, page = 7, 2, 128, 16
    width = 3008
    lens = np.array([20, 20, 20, -1, width - n + 1, width - n, 2900])
    ok = np.where((lens < 0) | (lens > width - n), 0, lens)
    p = kc.Pool(ssdv, B, Hkv, D, page, width)
    kh, vh = fill(p, ok, ok + n)
    p.table[1, 0] = p.cache.shape[0]
    p.table[2, 1] = -5
    p.table[6, 90] = 1 << 30
    p.table[0, 5] = -7  # never visited
    q, q64 = kc.rows((B, n, Hkv * G, D), BF16, 3)
    ws = ssdv.make_kv_workspace(n, Hkv * G, Hkv, D)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True, workspace=ws)
    assert ssdv.read_status(ws) == 12
    for b in (1, 2, 3, 4, 6):
        assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
    for b in (0, 5):
        ref = kc.attention(q64[b], kh[b], vh[b], int(lens[b]), n, D ** -0.5)
        tol, ltol = kc.bounds(*ref, D, BF16)
        assert (np.abs(out[b].double().cpu().numpy() - ref[0]) <= tol).all(), b
        assert (np.abs(lse[b].double().cpu().numpy() - ref[1]) <= ltol).all(), b
    again, alse = ssdv.kv_attention(p.cache, p.table, kc.ints(ok), q, n_q=kc.ints([n, 0, 0, n + 1, -1, n, 0]),
                                    return_lse=True, workspace=ws)
    assert ssdv.read_status(ws) == 13
    for b in (3, 4):
        assert bool(torch.isnan(again[b]).all()) and bool(torch.isnan(alse[b]).all()), b
    for b in (1, 2, 6):
        assert bool((again[b] == 0).all()) and bool((alse[b] == -np.inf).all()), b
    for b in (0, 5):
        ref = kc.attention(q64[b], kh[b], vh[b], int(lens[b]), n, D ** -0.5)
        tol, ltol = kc.bounds(*ref, D, BF16)
        assert (np.abs(again[b].double().cpu().numpy() - ref[0]) <= tol).all(), b


@ROWS
@pytest.mark.parametrize("scale,q_size", [(0.0, 1.0), (-0.3, 1.0), (3.0, 4.0), (1e-3, 1e3), (1.0, 1e-30)])
def test_scales(ssdv, n, G, scale, q_size):  # noqa: F811
    check(ssdv, 3, 1, G, 128, 16, BF16, n, [0, 40, 700], scale=scale, q_size=q_size)


@ROWS
@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales_with_masks(ssdv, n, G, scale):  # noqa: F811
    check(ssdv, 3, 2, G, 128, 32, BF16, n, [0, 130, 300], scale=scale, window=40)
    check(ssdv, 3, 2, G, 128, 32, BF16, n, [0, 130, 300], n_q=[n, 1, n - 1], scale=scale, past_only=True)


@ROWS
@pytest.mark.parametrize("length", [70, 126, 250])
def test_nan_values_alone(ssdv, n, G, length):  # noqa: F811
    """NaN values with finite keys: their 16 channels are NaN in the rows that see them, the others are right."""
    D = 128
    p = kc.Pool(ssdv, 1, 1, D, 16, length + n)
    k, k64 = kc.rows((1, length + n, 1, D), BF16, 1)
    v, v64 = kc.rows((1, length + n, 1, D), BF16, 2)
    gone = np.zeros((n, G, D), bool)
    for i, channel in ((1, 120), (2, 37), (n - 1, 3)):  # query i's own token, seen from it on
        v[0, length + i, 0, channel] = float("nan")
        group = slice(channel // 16 * 16, channel // 16 * 16 + 16)
        v64[0, length + i, 0, group] = 0
        gone[i:, :, group] = True
    p.append([0], k, v)
    q, q64 = kc.rows((1, n, G, D), BF16, 3)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints([length]), q, return_lse=True)
    o = out.double().cpu().numpy()[0]
    ref = kc.attention(q64[0], kc.held(k64)[0], kc.held(v64)[0], length, n, D ** -0.5)
    tol, ltol = kc.bounds(*ref, D, BF16)
    assert np.array_equal(np.isnan(o), gone)
    assert (np.abs(o - ref[0]) <= tol)[~gone].all()
    assert (np.abs(lse.double().cpu().numpy()[0] - ref[1]) <= ltol).all()


@ROWS
def test_graph_of_a_round(ssdv, n, G):  # noqa: F811
    """Append and attention captured once, replayed as the lengths advance."""
    B, Hkv, D = 3, 2, 128
    lens = np.array([0, 61, 730])
    p = kc.Pool(ssdv, B, Hkv, D, 32, 800)
    kh, vh = fill(p, lens, lens)
    kh, vh = [np.concatenate([x, np.zeros((B, 4 * n, Hkv, D))], 1) for x in (kh, vh)]
    q = torch.zeros(B, n, Hkv * G, D, dtype=BF16, device="cuda")
    k, v = (torch.zeros(B, n, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    at = kc.ints(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssdv.kv_append(p.cache, p.table, at, k, v)
        out, lse = ssdv.kv_attention(p.cache, p.table, at, q, return_lse=True)
    for step in range(3):
        q1, q64 = kc.rows(q.shape, BF16, 50 + step)
        k1, k64 = kc.rows(k.shape, BF16, 60 + step)
        v1, v64 = kc.rows(v.shape, BF16, 70 + step)
        q.copy_(q1), k.copy_(k1), v.copy_(v1)
        at.copy_(kc.ints(lens))
        graph.replay()
        for b in range(B):
            kh[b, lens[b]:lens[b] + n], vh[b, lens[b]:lens[b] + n] = kc.held(k64[b]), kc.held(v64[b])
        compare(p, q, q64, kh, vh, lens, np.full(B, n), BF16, out, lse)
        lens = lens + [1, n, 2]


@ROWS
def test_same_bits_again(ssdv, n, G):  # noqa: F811
    lens = np.array([1000, 3, 517, 2222, 0])
    p = kc.Pool(ssdv, 5, 2, 128, 64, 2300)
    fill(p, lens, lens + n)
    q, _ = kc.rows((5, n, 2 * G, 128), BF16, 3, 3.0)
    first, flse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
    for _ in range(4):
        out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
        assert torch.equal(out, first) and torch.equal(lse, flse)


@pytest.mark.parametrize("n,G", [(5, 4), (5, 8)])
def test_pool_past_32_bits(ssdv, n, G):  # noqa: F811
    H, D, page = 8, 128, 128
    n_pages = (5 << 30) // ssdv.lib().ssd_kv_page_bytes(H, D, page) - 1
    p = kc.Pool(ssdv, 1, H, D, page, 3 * page)
    p.cache = ssdv.make_kv_cache(n_pages, H, D, page, device="cuda")
    p.table = kc.ints([[n_pages - 1, 3, n_pages - 2]])
    lens = np.array([330])
    kh, vh = fill(p, lens, lens + n)
    q, q64 = kc.rows((1, n, H * G, D), BF16, 3)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
    compare(p, q, q64, kh, vh, lens, np.full(1, n), BF16, out, lse)
