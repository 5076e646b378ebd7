"""Attention over the 4-bit cache on the GPU, against the definition in 64 bits
over the values the cache holds (error bounds: kv_common.bounds)."""
import numpy as np
import pytest
import torch

import gpu_common as gc
import kv_common as kc

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssdv():
    return gc.cuda_lib()


def fill(p, lens, total, dtype=BF16, seed=1, v_size=1.0):
    """Keys and values of `total[b]` tokens per request, in the pool; returns what it holds."""
    n = max(1, int(max(total)))
    k, k64 = kc.rows((p.B, n, p.H, p.D), dtype, seed)
    v, v64 = kc.rows((p.B, n, p.H, p.D), dtype, seed + 1, v_size)
    p.append(np.zeros(p.B), k, v, n_new=total)
    return kc.held(k64), kc.held(v64)


def compare(p, q, q64, kh, vh, lens, n_q, dtype, out, lse, scale=None, window=0, past_only=False, what=""):
    scale = p.D ** -0.5 if scale is None else scale
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(p.B):
        ref = kc.attention(q64[b], kh[b], vh[b], int(lens[b]), int(n_q[b]), scale, window, past_only)
        tol, ltol = kc.bounds(*ref, p.D, dtype)
        gone = ref[4] == 0
        assert (out[b][gone] == 0).all() and (lse[b][gone] == -np.inf).all(), (what, b)
        err = np.abs(out[b] - ref[0])
        assert (err <= tol)[~gone].all(), (what, b, float(np.nanmax(err / tol)), int(np.isnan(err).sum()))
        lerr = np.abs(lse[b][~gone] - ref[1][~gone])
        assert (lerr <= ltol[~gone]).all(), (what, b, float((lerr / ltol[~gone]).max()))


def check(ssdv, B, Hkv, G, D, page, dtype, n, lens, n_q=None, window=0, past_only=False, scale=None, seed=1, fill_byte=0xFF,
          q_size=1.0):
    lens = np.asarray(lens)
    nq = np.full(B, n) if n_q is None else np.asarray(n_q)
    p = kc.Pool(ssdv, B, Hkv, D, page, int(lens.max()) + n, seed=seed, fill=fill_byte)
    kh, vh = fill(p, lens, lens if past_only else lens + nq, seed=seed)
    q, q64 = kc.rows((B, n, Hkv * G, D), dtype, seed + 7, q_size)
    ws = ssdv.make_kv_workspace(n, Hkv * G, Hkv, D)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, n_q=None if n_q is None else kc.ints(n_q), scale=scale,
                                 window=window, past_only=past_only, return_lse=True, workspace=ws)
    assert ssdv.read_status(ws) == 0
    compare(p, q, q64, kh, vh, lens, nq, dtype, out, lse, scale, window, past_only)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,Hkv,page", [(64, 2, 16), (128, 2, 64), (256, 1, 32)])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 8), (5, 4), (3, 3), (5, 8), (9, 8), (32, 1), (2, 13), (7, 16)])
def test_shapes(ssdv, dtype, D, Hkv, page, n, G):
    check(ssdv, 3, Hkv, G, D, page, dtype, n, [0, 77, 190])


@pytest.mark.parametrize("page", [16, 48, 64, 128])
@pytest.mark.parametrize("past_only", [False, True])
def test_lengths(ssdv, page, past_only):
    """Every length around a block, a page and a tile's end, zero and one among them."""
    lens = [0, 1, 2, 14, 15, 16, 17, 31, 32, 47, 48, 49, 59, 60, 61, 63, 64, 65, 95, 127, 128, 129, 255, 256, 300]
    check(ssdv, len(lens), 1, 2, 64, page, BF16, 4, lens, past_only=past_only)
    check(ssdv, len(lens), 1, 2, 128, page, BF16, 1, lens, past_only=past_only)


@pytest.mark.parametrize("window", [1, 2, 3, 16, 63, 64, 65, 100, 1 << 20])
@pytest.mark.parametrize("past_only", [False, True])
def test_windows(ssdv, window, past_only):
    """Windows from one token; over the past alone a small one leaves later rows empty."""
    check(ssdv, 4, 2, 4, 128, 32, BF16, 6, [0, 3, 130, 257], window=window, past_only=past_only)
    check(ssdv, 2, 1, 1, 64, 16, F32, 6, [5, 400], window=window, past_only=past_only)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged_queries(ssdv, D):
    """Per-request query counts, none among them."""
    check(ssdv, 6, 2, 8, D, 64, BF16, 9, [10, 0, 200, 333, 64, 0], n_q=[9, 1, 0, 4, 7, 0])
    check(ssdv, 4, 2, 3, D, 64, F32, 9, [10, 0, 200, 0], n_q=[1, 0, 9, 5], past_only=True)


@pytest.mark.parametrize("G,n,dtype", [(8, 5, BF16), (4, 2, F32), (1, 1, BF16), (16, 32, BF16)])
def test_long_context(ssdv, G, n, dtype):
    check(ssdv, 1, 1, G, 128, 64, dtype, n, [9001])
    check(ssdv, 3, 2, G, 64, 16, dtype, min(n, 3), [5003, 17, 1200])


def test_many_requests(ssdv):
    g = np.random.default_rng(2)
    B = 300
    check(ssdv, B, 2, 4, 64, 16, BF16, 3, g.integers(0, 90, B), n_q=g.integers(0, 4, B))


def test_most_heads_and_queries(ssdv):
    """128 query heads a kv head and 32 query tokens: 4096 rows share each key."""
    check(ssdv, 1, 1, 128, 64, 16, BF16, 32, [70])


@pytest.mark.parametrize("scale,q_size", [(0.0, 1.0), (-0.3, 1.0), (3.0, 4.0), (1e-3, 1e3), (1.0, 1e-30)])
def test_scales(ssdv, scale, q_size):
    """Uniform weights, negative scale, scores in the thousands (one token decides), queries far from one."""
    for dtype in (BF16, F32):
        check(ssdv, 2, 1, 4, 128, 16, dtype, 3, [40, 200], scale=scale, q_size=q_size)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_query_strides(ssdv, dtype):
    B, n, Hkv, G, D = 2, 5, 2, 4, 64
    lens = np.array([33, 120])
    p = kc.Pool(ssdv, B, Hkv, D, 16, 130)
    kh, vh = fill(p, lens, lens + n)
    q, q64 = kc.rows((B, n, Hkv * G, D), dtype, 3)
    flat = torch.zeros(q.numel() * 2 + 1, dtype=dtype, device="cuda")
    odd = flat[1:1 + q.numel()].view(q.shape).copy_(q)
    wide = flat.new_zeros(B, n, 3, Hkv * G, D)
    wide[:, :, 1] = q
    first = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    for form in (odd, wide[:, :, 1], first):
        out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), form, return_lse=True)
        compare(p, q, q64, kh, vh, lens, np.full(B, n), dtype, out, lse)


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (128, F32), (256, BF16)])
def test_nan_and_inf_in_masked_places(ssdv, D, dtype):
    """A token whose key and value are NaN or infinite changes nothing for the rows that do not see it: drafts after
    a row, tokens before a window, rejected drafts past the length."""
    B, Hkv, G, n, T = 2, 1, 4, 5, 150
    lens = np.array([97, 126])
    for window in (0, 40):
        p = kc.Pool(ssdv, B, Hkv, D, 16, T + 16, fill=0xFF)
        k, k64 = kc.rows((B, T, Hkv, D), BF16, 1)
        v, v64 = kc.rows((B, T, Hkv, D), BF16, 2)
        bad = [lens + 2, lens + n, lens + n + 1, lens - 60]  # seen by rows 2.. only; past the end; before the window
        for b in range(B):
            for j, at in enumerate(bad):
                if j == 3 and not window:
                    continue
                for x, x64 in ((k, k64), (v, v64)):
                    x[b, at[b], 0, j] = float("nan") if j != 1 else float("inf")
                    x64[b, at[b], 0, j] = np.nan if j != 1 else np.inf
        p.append([0, 0], k, v)
        kh, vh = kc.held(k64), kc.held(v64)
        q, q64 = kc.rows((B, n, G, D), dtype, 3)
        out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, window=window, return_lse=True)
        o = out.double().cpu().numpy()
        assert np.isnan(o[:, 2:]).all() and np.isnan(lse[:, 2:].cpu().numpy()).all()
        for i in range(2):
            compare(p, q[:, i:i + 1], q64[:, i:i + 1], kh, vh, lens + i, np.ones(B), dtype, out[:, i:i + 1], lse[:, i:i + 1],
                    window=window)


def test_nan_value_alone(ssdv):
    """A NaN value with a finite key: its 16 channels are NaN in the rows that see it, the others are right."""
    D, lens, n = 128, np.array([70]), 4
    p = kc.Pool(ssdv, 1, 1, D, 16, 80)
    k, k64 = kc.rows((1, 74, 1, D), BF16, 1)
    v, v64 = kc.rows((1, 74, 1, D), BF16, 2)
    v[0, 72, 0, 37] = float("nan")
    p.append([0], k, v)
    q, q64 = kc.rows((1, n, 2, D), BF16, 3)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
    o = out.double().cpu().numpy()
    assert np.isnan(o[0, 2:, :, 32:48]).all()
    o[0, 2:, :, 32:48] = 0
    v64[0, 72, 0, 32:48] = 0
    vh = kc.held(v64)
    ref = kc.attention(q64[0], kc.held(k64)[0], vh[0], 70, n, D ** -0.5)
    tol, ltol = kc.bounds(*ref, D, BF16)
    ref[0][2:, :, 32:48] = 0
    assert (np.abs(o[0] - ref[0]) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy()[0] - ref[1]) <= ltol).all()


def test_errors_stay_with_their_request(ssdv):
    B, Hkv, G, D, page, n = 6, 2, 4, 128, 16, 3
    lens = np.array([20, 20, 20, -1, 46, 45])
    ok = np.array([20, 20, 20, 0, 40, 45])
    p = kc.Pool(ssdv, B, Hkv, D, page, 48)
    kh, vh = fill(p, ok, ok + n)
    p.table[1, 0] = p.cache.shape[0]
    p.table[2, 1] = -5
    p.table[0, 2] = -7  # never visited
    q, q64 = kc.rows((B, n, Hkv * G, D), BF16, 3)
    ws = ssdv.make_kv_workspace(n, Hkv * G, Hkv, D)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True, workspace=ws)
    assert ssdv.read_status(ws) == 12
    for b in (1, 2, 3, 4):
        assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
    for b in (0, 5):
        ref = kc.attention(q64[b], kh[b], vh[b], int(lens[b]), n, D ** -0.5)
        tol, ltol = kc.bounds(*ref, D, BF16)
        assert (np.abs(out[b].double().cpu().numpy() - ref[0]) <= tol).all()
    again, _ = ssdv.kv_attention(p.cache, p.table, kc.ints(ok), q, n_q=kc.ints([3, 0, 0, 4, -1, 3]), return_lse=True,
                                 workspace=ws)
    assert ssdv.read_status(ws) == 13
    assert torch.equal(again[0], out[0]) and bool(torch.isnan(again[3]).all()) and bool(torch.isnan(again[4]).all())
    assert bool((again[1] == 0).all())


def test_same_bits_again_and_on_another_stream(ssdv):
    lens = np.array([1000, 3, 517, 2222])
    p = kc.Pool(ssdv, 4, 2, 128, 64, 2300)
    fill(p, lens, lens + 5)
    q, _ = kc.rows((4, 5, 16, 128), BF16, 3)
    at = kc.ints(lens)
    first, flse = ssdv.kv_attention(p.cache, p.table, at, q, return_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side, None):
        out, lse = ssdv.kv_attention(p.cache, p.table, at, q, return_lse=True, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(lse, flse)


def test_graph_of_a_round(ssdv):
    """Append and attention captured once, replayed as the lengths advance."""
    B, n, Hkv, G, D = 3, 4, 2, 4, 128
    lens = np.array([0, 61, 130])
    p = kc.Pool(ssdv, B, Hkv, D, 32, 200)
    total, q = lens.max() + 3 * n, torch.empty(B, n, Hkv * G, D, dtype=BF16, device="cuda")
    kh, vh = fill(p, lens, lens)
    kh, vh = [np.concatenate([x, np.zeros((B, 4 * n, Hkv, D))], 1) for x in (kh, vh)]
    k, v = torch.empty(B, n, Hkv, D, dtype=BF16, device="cuda"), torch.empty(B, n, Hkv, D, dtype=BF16, device="cuda")
    at = kc.ints(lens)
    for x in (q, k, v):
        x.zero_()
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
        lens = lens + [1, 4, 2]
    assert total <= 200


def test_parts_join_by_lse(ssdv):
    """Attention over the past alone, joined by its log-sum-exp to attention over the new tokens' own keys, is the
    attention over all of them."""
    B, n, Hkv, G, D = 2, 3, 1, 4, 64
    lens = np.array([50, 0])
    p = kc.Pool(ssdv, B, Hkv, D, 16, 64)
    kh, vh = fill(p, lens, lens + n)
    q, q64 = kc.rows((B, n, G, D), F32, 3)
    past, plse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, past_only=True, return_lse=True)
    both, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
    for b in range(B):
        own = kc.attention(q64[b], kh[b, lens[b]:], vh[b, lens[b]:], 0, n, D ** -0.5)
        a, c = plse[b].double().cpu().numpy(), own[1]
        z = np.logaddexp(a, c)
        y = np.exp(a - z)[..., None] * past[b].double().cpu().numpy() + np.exp(c - z)[..., None] * own[0]
        ref = kc.attention(q64[b], kh[b], vh[b], int(lens[b]), n, D ** -0.5)
        tol, ltol = kc.bounds(*ref, D, F32)
        assert (np.abs(z - lse[b].double().cpu().numpy()) <= 2 * ltol).all()
        assert (np.abs(y - both[b].double().cpu().numpy()) <= 3 * tol).all()


def test_pool_past_32_bits(ssdv):
    H, D, page = 8, 128, 128
    n_pages = (5 << 30) // ssdv.lib().ssd_kv_page_bytes(H, D, page) - 1
    p = kc.Pool(ssdv, 1, H, D, page, 3 * page)
    p.cache = ssdv.make_kv_cache(n_pages, H, D, page, device="cuda")
    p.table = kc.ints([[n_pages - 1, 3, n_pages - 2]])
    lens = np.array([330])
    kh, vh = fill(p, lens, lens + 2)
    q, q64 = kc.rows((1, 2, 16, D), BF16, 3)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
    compare(p, q, q64, kh, vh, lens, np.full(1, 2), BF16, out, lse)


def test_query_strides_of_many_rows(ssdv):
    B, n, Hkv, G, D = 2, 5, 2, 8, 128
    lens = np.array([33, 300])
    p = kc.Pool(ssdv, B, Hkv, D, 16, 310)
    kh, vh = fill(p, lens, lens + n)
    q, q64 = kc.rows((B, n, Hkv * G, D), BF16, 3)
    odd = torch.zeros(q.numel() + 1, dtype=BF16, device="cuda")[1:].view(q.shape).copy_(q)
    wide = q.new_zeros(B, n, 3, Hkv * G, D)
    wide[:, :, 1] = q
    padded = q.new_zeros(B, n, Hkv * G, D + 4)[..., :D].copy_(q)
    first = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    for form in (odd, wide[:, :, 1], padded, first):
        out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), form, return_lse=True)
        compare(p, q, q64, kh, vh, lens, np.full(B, n), BF16, out, lse)


@pytest.mark.parametrize("n,G,past_only", [(1, 4, False), (5, 8, False), (5, 13, True), (4, 6, True)])
def test_uneven_shares(ssdv, n, G, past_only):
    # many beginnings of rows next to long ones: shares that hold only beginnings, rows split at every place
    rng = np.random.default_rng(n)
    lens = np.concatenate([np.zeros(40, int), rng.integers(1, 4, 60), rng.integers(1, 700, 180), [3001, 1, 0, 1999]])
    rng.shuffle(lens)
    n_q = rng.integers(0, n + 1, lens.size)
    check(ssdv, lens.size, 2, G, 128, 32, BF16, n, lens, n_q=n_q, past_only=past_only)
