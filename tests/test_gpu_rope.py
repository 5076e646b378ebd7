"""Norms and rotation of queries and keys on the GPU against the formula in 64
bits (bounds: round_common.rope_bound)."""
import numpy as np
import pytest
import torch

import gpu_common as gc
import kv_common as kc
import round_common as rc

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
LENGTH = 13


@pytest.fixture(scope="module")
def ssdv():
    return gc.cuda_lib()


def freqs(rot, theta=500000.0):
    return torch.from_numpy(theta ** (-np.arange(rot // 2) / (rot // 2))).float().cuda() if rot else None


def compare(q, x, lens, news, weight, eps, freq, interleaved, dtype):
    """Result q of rows x (64 bits)."""
    q = q.double().cpu().numpy()
    w = None if weight is None else weight.cpu().numpy()
    f = None if freq is None else freq.cpu().numpy()
    for b in range(x.shape[0]):
        m = int(news[b])
        y, size = rc.rope(x[b, :m], int(lens[b]) + np.arange(m), w, eps, f, interleaved)
        err, tol = np.abs(q[b, :m] - y), rc.rope_bound(y, size, dtype)
        assert (err <= tol).all(), (b, float(np.nanmax(err / tol)))
        assert (q[b, m:] == 0).all()


def check(ssdv, B, n, H, Hkv, D, rot, dtype, lens, news=None, norm=True, interleaved=False, eps=1e-6, seed=1, theta=500000.0,
          size=1.0):
    q, q64 = kc.rows((B, n, H, D), dtype, seed, size)
    k, k64 = kc.rows((B, n, Hkv, D), dtype, seed + 1, size)
    g = torch.Generator().manual_seed(seed)
    qw, kw = ((torch.randn(D, generator=g).cuda(), torch.randn(D, generator=g).cuda()) if norm else (None, None))
    freq = freqs(rot, theta)
    ws = ssdv.make_kv_workspace()
    oq, ok = ssdv.qk_norm_rope(q, k, kc.ints(lens), qw, kw, freq, eps, interleaved,
                               n_new=None if news is None else kc.ints(news), workspace=ws)
    assert ssdv.read_status(ws) == 0
    news = np.full(B, n) if news is None else news
    compare(oq, q64, lens, news, qw, eps, freq, interleaved, dtype)
    compare(ok, k64, lens, news, kw, eps, freq, interleaved, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rots", [(64, (0, 16, 32, 48, 64)), (128, (0, 16, 80, 128)), (256, (0, 64, 176, 256))])
def test_shapes(ssdv, D, rots, interleaved, dtype):
    for rot in rots:
        for H, Hkv in ((1, 1), (5, 2), (32, 8), (3, 0), (17, 17)):
            if Hkv:
                check(ssdv, 3, 4, H, Hkv, D, rot, dtype, [0, 9, 1000], interleaved=interleaved, norm=rot % 32 == 0)


def test_queries_alone_and_one_norm(ssdv):
    q, q64 = kc.rows((2, 3, 4, 64), BF16, 5)
    k, k64 = kc.rows((2, 3, 2, 64), BF16, 6)
    lens, w, f = np.array([3, 70000]), torch.randn(64).cuda(), freqs(64)
    oq, ok = ssdv.qk_norm_rope(q, None, kc.ints(lens), w, None, f)
    assert ok is None
    compare(oq, q64, lens, [3, 3], w, 1e-6, f, False, BF16)
    oq, ok = ssdv.qk_norm_rope(q, k, kc.ints(lens), None, w, f)
    compare(oq, q64, lens, [3, 3], None, 1e-6, f, False, BF16)
    compare(ok, k64, lens, [3, 3], w, 1e-6, f, False, BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_positions(ssdv, dtype):
    """Angles of positions up to 2^30, of frequencies down to 1e-8 and above one turn a token."""
    lens = np.array([0, 1, 4097, 131071, 1 << 20, (1 << 24) + 1, 999999937, (1 << 30) - 4])
    check(ssdv, 8, 4, 4, 2, 128, 128, dtype, lens, theta=1e8)
    q, q64 = kc.rows((8, 4, 2, 64), dtype, 2)
    freq = torch.tensor([0.0, 1.0, -1.0, 6.2831855, 3.1415927, 100.25, -0.3, 1e-8] + [1e-3] * 24).cuda()
    # (64-bit angles of 1e11 radians are themselves off by 1e-5: positions below 2^24 for the fast ones)
    lens = np.minimum(lens, 1 << 23)
    oq, _ = ssdv.qk_norm_rope(q, None, kc.ints(lens), inv_freq=freq)
    compare(oq, q64, lens, np.full(8, 4), None, 0, freq, False, dtype)


def test_ragged_and_padded(ssdv):
    """Rows past a request's count are not read (NaN there) and become zero."""
    news = np.array([0, 1, 5, 3])
    lens = np.array([7, 0, 100, 31])
    q, q64 = kc.rows((4, 5, 6, 128), BF16, 3)
    k, k64 = kc.rows((4, 5, 2, 128), BF16, 4)
    for b in range(4):
        q[b, news[b]:] = float("nan")
        k[b, news[b]:] = float("nan")
    w, f = torch.randn(128).cuda(), freqs(128)
    oq, ok = ssdv.qk_norm_rope(q, k, kc.ints(lens), w, w, f, n_new=kc.ints(news))
    compare(oq, q64, lens, news, w, 1e-6, f, False, BF16)
    compare(ok, k64, lens, news, w, 1e-6, f, False, BF16)
    check(ssdv, 4, 5, 6, 2, 64, 32, F32, lens, news=news, interleaved=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_in_place(ssdv, dtype):
    """Slices of one projection, unaligned rows, heads before tokens; in place in all of them."""
    B, n, H, Hkv, D = 2, 3, 4, 2, 64
    lens, f, w = np.array([5, 900]), freqs(32), torch.randn(D).cuda()
    x, x64 = kc.rows((B, n, H + 2 * Hkv, D), dtype, 8)
    flat = torch.zeros(x.numel() + 1, dtype=dtype, device="cuda")
    odd = flat[1:].view(x.shape).copy_(x)
    turned = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    for form in (x.clone(), odd, turned):
        before = form.clone()
        q, k = form[:, :, :H], form[:, :, H:H + Hkv]
        oq, ok = ssdv.qk_norm_rope(q, k, kc.ints(lens), w, w, f)
        compare(oq, x64[:, :, :H], lens, [n, n], w, 1e-6, f, False, dtype)
        compare(ok, x64[:, :, H:H + Hkv], lens, [n, n], w, 1e-6, f, False, dtype)
        assert torch.equal(form, before)
        ssdv.qk_norm_rope(q, k, kc.ints(lens), w, w, f, out=(q, k))
        assert torch.equal(q, oq) and torch.equal(k, ok)
        assert torch.equal(form[:, :, H + Hkv:], before[:, :, H + Hkv:])


def test_values(ssdv):
    """Zero rows, large and small rows, and an infinity or a NaN that stays in its own row."""
    q = torch.zeros(1, 1, 6, 64, device="cuda")
    q[0, 0, 1], q[0, 0, 2], q[0, 0, 3, 5], q[0, 0, 4, 5] = 1e18, 1e-18, float("nan"), 1.0
    f = freqs(64)
    w = torch.ones(64, device="cuda")
    out, _ = ssdv.qk_norm_rope(q, None, kc.ints([3]), w, None, f, eps=0.0)
    out = out.cpu().double().numpy()[0, 0]
    assert np.isnan(out[0]).all() and np.isnan(out[3]).all() and np.isnan(out[5]).all()  # 0 / 0 without eps
    for j, value in ((1, 1e18), (2, 1e-18)):
        y, size = rc.rope(np.full((1, 1, 64), np.float64(np.float32(value))), np.array([3]), np.ones(64), 0.0, f.cpu().numpy(), False)
        assert (np.abs(out[j] - y[0, 0]) <= rc.rope_bound(y, size, F32)[0, 0]).all()
    out, _ = ssdv.qk_norm_rope(q, None, kc.ints([3]), w, None, f)
    assert (out[0, 0, 0] == 0).all() and torch.isfinite(out[0, 0, 4]).all()


def test_bad_lengths(ssdv):
    q, q64 = kc.rows((5, 3, 2, 64), BF16, 1)
    lens, news = np.array([-1, 4, (1 << 30) - 2, 4, 9]), np.array([3, 4, 3, -1, 2])
    ws = ssdv.make_kv_workspace()
    f = freqs(64)
    out, _ = ssdv.qk_norm_rope(q, None, kc.ints(lens), inv_freq=f, n_new=kc.ints(news), workspace=ws)
    assert ssdv.read_status(ws) == LENGTH
    assert torch.isnan(out[:4]).all()
    compare(out[4:], q64[4:], lens[4:], news[4:], None, 0, f, False, BF16)


def test_capture_and_stream(ssdv):
    q, q64 = kc.rows((2, 3, 4, 128), BF16, 1)
    k, k64 = kc.rows((2, 3, 2, 128), BF16, 2)
    lens, f = kc.ints([5, 77]), freqs(128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = ssdv.qk_norm_rope(q, k, lens, inv_freq=f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = ssdv.qk_norm_rope(q, k, lens, inv_freq=f)
    lens += 1
    graph.replay()
    compare(b[0], q64, [6, 78], [3, 3], None, 0, f, False, BF16)
    compare(a[1], k64, [5, 77], [3, 3], None, 0, f, False, BF16)


def test_many_tokens(ssdv):
    """More CTAs than run at a time, ragged, against the rows of single calls."""
    B, n = 3, 2500
    q, q64 = kc.rows((B, n, 3, 64), BF16, 1)
    k, k64 = kc.rows((B, n, 1, 64), BF16, 2)
    news, lens, f = np.array([2500, 17, 1999]), np.array([0, 5, 100000]), freqs(64)
    oq, ok = ssdv.qk_norm_rope(q, k, kc.ints(lens), inv_freq=f, n_new=kc.ints(news))
    compare(oq, q64, lens, news, None, 0, f, False, BF16)
    compare(ok, k64, lens, news, None, 0, f, False, BF16)
