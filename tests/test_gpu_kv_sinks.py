"""Attention within a window with first tokens that stay visible, against the
definition in 64 bits (error bounds: kv_common.bounds)."""
import numpy as np
import pytest
import torch

import gpu_common as gc
import kv_common as kc
import round_common as rc
from test_gpu_kv_attention import fill

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PAGE = 12


@pytest.fixture(scope="module")
def ssdv():
    return gc.cuda_lib()


def visible(length, i, window, sinks, past_only):
    t = np.arange(length if past_only else length + i + 1)
    return t[(t > length + i - window) | (t < sinks)]


def compare(p, q64, kh, vh, lens, n_q, dtype, out, lse, window, sinks, past_only=False, scale=None):
    scale = p.D ** -0.5 if scale is None else scale
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(p.B):
        ref, _ = rc.attend(q64[b], kh[b], vh[b],
                        lambda i: visible(int(lens[b]), i, window, sinks, past_only) if i < n_q[b] else np.arange(0), scale)
        tol, ltol = kc.bounds(*ref, p.D, dtype)
        gone = ref[4] == 0
        assert (out[b][gone] == 0).all() and (lse[b][gone] == -np.inf).all(), b
        err = np.abs(out[b] - ref[0])
        assert (err <= tol)[~gone].all(), (b, float(np.nanmax(err / tol)), int(np.isnan(err).sum()))
        lerr = np.abs(lse[b][~gone] - ref[1][~gone])
        assert (lerr <= ltol[~gone]).all(), (b, float((lerr / ltol[~gone]).max()))


def check(ssdv, B, Hkv, G, D, page, dtype, n, lens, window, sinks, n_q=None, past_only=False, sharp=False):
    lens = np.asarray(lens)
    nq = np.full(B, n) if n_q is None else np.asarray(n_q)
    p = kc.Pool(ssdv, B, Hkv, D, page, int(lens.max()) + n, fill=0xFF)
    total = lens if past_only else lens + nq
    m = max(1, int(total.max()))
    k, k64 = kc.rows((B, m, Hkv, D), dtype, 1)
    v, v64 = kc.rows((B, m, Hkv, D), dtype, 2)
    q, q64 = kc.rows((B, n, Hkv * G, D), dtype, 8)
    if sharp:  # the first tokens draw the weight, their values are zero
        k[:, :4], v[:, :4] = q[:, :1, :Hkv] * 2, 0
        k64, v64 = k.double().cpu().numpy(), v.double().cpu().numpy()
    p.append(np.zeros(B), k, v, n_new=total)
    ws = ssdv.make_kv_workspace(n, Hkv * G, Hkv, D)
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, n_q=None if n_q is None else kc.ints(n_q), window=window,
                                 sinks=sinks, past_only=past_only, return_lse=True, workspace=ws)
    assert ssdv.read_status(ws) == 0
    compare(p, q64, kc.held(k64), kc.held(v64), lens, nq, dtype, out, lse, window, sinks, past_only)
    return p, q, out, lse


@pytest.mark.parametrize("past_only", [False, True])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 129, 300])
@pytest.mark.parametrize("sinks", [1, 4, 16, 64, 65, 128, 130, 1000])
def test_windows_and_sinks(ssdv, window, sinks, past_only):
    """Sinks inside the window, beside it and far before it; the shared and the matrix-instruction forms of few rows."""
    lens = [0, 1, 3, 64, 65, 127, 130, 257, 400, 700]
    check(ssdv, len(lens), 1, 4, 128, 32, BF16, 3, lens, window, sinks, past_only=past_only)
    check(ssdv, len(lens), 1, 5, 128, 16, BF16, 4, lens, window, sinks, past_only=past_only)  # 20 rows


@pytest.mark.parametrize("dtype,D,Hkv,G,n", [(BF16, 64, 2, 3, 5), (BF16, 256, 2, 4, 5), (F32, 64, 2, 1, 4), (F32, 128, 1, 8, 3),
                                             (F32, 256, 1, 2, 2), (BF16, 128, 2, 1, 1), (BF16, 128, 2, 8, 5),
                                             (BF16, 128, 1, 16, 9), (BF16, 128, 1, 6, 8)])
def test_types_heads_and_rows(ssdv, dtype, D, Hkv, G, n):
    for window, sinks in ((100, 3), (5, 70), (257, 129)):
        check(ssdv, 4, Hkv, G, D, 48, dtype, n, [0, 90, 333, 1500], window, sinks)
        check(ssdv, 4, Hkv, G, D, 64, dtype, n, [0, 90, 333, 1500], window, sinks, n_q=[n, 0, 1, n // 2], past_only=True)


@pytest.mark.parametrize("G,n", [(1, 1), (4, 5), (8, 8)])
def test_long_contexts(ssdv, G, n):
    check(ssdv, 2, 1, G, 128, 64, BF16, n, [20011, 9001], 4096, 4)
    check(ssdv, 1, 2, G, 128, 128, BF16, n, [30000], 1, 200)


@pytest.mark.parametrize("G", [2, 8])
def test_sinks_that_draw_the_weight(ssdv, G):
    """Large scores and values of zero at the first tokens: what remains is the window's small weights."""
    check(ssdv, 3, 2, G, 128, 64, BF16, 5, [50, 600, 1500], 500, 4, sharp=True)
    check(ssdv, 3, 2, G, 64, 16, BF16, 5, [50, 600, 1500], 500, 4, sharp=True)


@pytest.mark.parametrize("G", [2, 8])
def test_many_requests_share_tiles_unevenly(ssdv, G):
    g = np.random.default_rng(5)
    B = 200
    check(ssdv, B, 2, G, 128, 16, BF16, 3, g.integers(0, 900, B), 130, 20, n_q=g.integers(0, 4, B))


def test_no_sinks_and_no_window(ssdv):
    """Without a window sinks change nothing, and without sinks the window's call is what it was."""
    lens = np.array([40, 500])
    p = kc.Pool(ssdv, 2, 2, 128, 16, 505)
    fill(p, lens, lens + 5)
    q, _ = kc.rows((2, 5, 16, 128), BF16, 3)
    a = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True)
    b = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, return_lse=True, sinks=100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    lib, out = ssdv.lib(), torch.empty_like(q)
    c, _, _ = ssdv._kv_cache(p.cache, p.table, 2)
    qp, qs = ssdv._kv_rows(q, "q", None, 128, 0)
    ws = ssdv.make_kv_workspace(5, 16, 2, 128)
    assert lib.ssd_kv_attention(c, kc.ints(lens).data_ptr(), None, qp, qs, 0, 2, 5, 16, 128 ** -0.5, 77, 0, out.data_ptr(),
                                None, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, window=77, sinks=0))


@pytest.mark.parametrize("D,G,n,dtype", [(64, 4, 5, BF16), (128, 2, 5, BF16), (128, 8, 5, BF16), (128, 2, 5, F32)])
def test_nan_between_sinks_and_window(ssdv, D, G, n, dtype):
    """NaN in tokens that no row sees, or only some rows, or a sink that all see."""
    B, T, window, sinks = 3, 300, 50, 5
    lens = np.array([200, 255, 290])
    p = kc.Pool(ssdv, B, 1, D, 16, T + 16, fill=0xFF)
    k, k64 = kc.rows((B, T + 5, 1, D), BF16, 1)
    v, v64 = kc.rows((B, T + 5, 1, D), BF16, 2)
    q, q64 = kc.rows((B, n, G, D), dtype, 3)
    clean_k, clean_v = k64.copy(), v64.copy()
    for b in range(B):
        for t in (5, 6, 100, int(lens[b]) - window, int(lens[b]) + n):  # seen by no row
            k[b, t], v[b, t] = float("nan"), float("nan")
            clean_k[b, t] = clean_v[b, t] = 0
    only = int(lens[1]) - window + 1  # row 0 of request 1 sees it
    v[1, only] = float("nan")
    p.append(np.zeros(B), k, v, n_new=np.minimum(lens + n + 1, T + 5))
    out, lse = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, window=window, sinks=sinks, return_lse=True)
    assert torch.isnan(out[1, 0]).all()
    clean_v[1, only] = 0
    kh, vh = kc.held(clean_k), kc.held(clean_v)
    ref, _ = rc.attend(q64[1], kh[1], vh[1], lambda i: visible(int(lens[1]), i, window, sinks, False), D ** -0.5)
    out[1, 0] = torch.from_numpy(ref[0][0]).to(out)  # (its NaN is right)
    compare(p, q64, kh, vh, lens, np.full(B, n), dtype, out, lse, window, sinks)
    v[2, 3] = float("nan")  # a sink
    p.append(np.zeros(B), k, v, n_new=np.minimum(lens + n + 1, T + 5))
    out = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, window=window, sinks=sinks)
    assert torch.isnan(out[2]).all() and not torch.isnan(out[0]).any()


@pytest.mark.parametrize("G", [2, 8])
def test_pages_between_sinks_and_window_may_be_gone(ssdv, G):
    """Bad page numbers where no row looks are not looked at; a sink's bad page is the request's loss."""
    lens, n = np.array([700, 650]), 3
    p, q, out, lse = check(ssdv, 2, 1, G, 128, 16, BF16, n, lens, 100, 4)
    ws = ssdv.make_kv_workspace(n, G, 1, 128)
    p.table[:, 1:30] = -1
    again = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, window=100, sinks=4, workspace=ws)
    assert ssdv.read_status(ws) == 0 and torch.equal(again, out)
    p.table[1, 0] = 1 << 30
    again = ssdv.kv_attention(p.cache, p.table, kc.ints(lens), q, window=100, sinks=4, workspace=ws)
    assert ssdv.read_status(ws) == PAGE and torch.isnan(again[1]).all() and torch.equal(again[0], out[0])
