"""The 4-bit key/value cache on the GPU: what is written, read back, against the
definition in 64 bits.  Both are exact, so every comparison is equality."""
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


@pytest.mark.parametrize("D,H,page,dtype", [(64, 3, 16, BF16), (64, 1, 48, F32), (128, 2, 64, BF16), (128, 8, 16, F32),
                                            (256, 2, 32, BF16), (256, 1, 128, F32)])
@pytest.mark.parametrize("start,n", [(0, 1), (0, 16), (15, 1), (7, 5), (13, 33), (31, 100)])
def test_round_trip(ssdv, D, H, page, dtype, start, n):
    B = 3
    starts = [start, start + 1, 2 * start]
    p = kc.Pool(ssdv, B, H, D, page, 2 * start + n + 2, seed=n)
    k, k64 = kc.rows((B, n, H, D), dtype, 1)
    v, v64 = kc.rows((B, n, H, D), dtype, 2)
    p.append(starts, k, v)
    for out in (F32, BF16):
        rk, rv = p.read(starts, n, out)
        np.testing.assert_array_equal(rk, kc.held(k64))
        np.testing.assert_array_equal(rv, kc.held(v64))
    assert ssdv.read_status(ssdv.kv_workspace()) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_special_values(ssdv, dtype):
    """Zeros, subnormal scales, the cap, infinities, NaN, and exact ties."""
    D, n = 64, 16
    x = torch.zeros(1, n, 1, D)
    g = torch.Generator().manual_seed(5)
    base = torch.randn(D, generator=g)
    for t, size in enumerate([0.0, 1e-30, 2.0 ** -19, 7 * 2.0 ** -18, 7 * 1.5 * 2.0 ** -17, 3e-5, 1e-3, 1.0, 300.0, 1680.0,
                              1737.0, 5000.0, 1e30]):
        x[0, t, 0] = base * size
    x[0, 13, 0] = torch.arange(D) % 15 - 7.0  # scale 1: whole numbers
    x[0, 14, 0] = (torch.arange(D) % 14 - 6.5)  # halves: ties to even wherever the scale is a power of two
    x[0, 14, 0, ::16] = 7.0
    x[0, 15, 0] = base
    x[0, 15, 0, 3] = float("nan")
    x[0, 15, 0, 20] = float("inf")
    x[0, 15, 0, 40] = -float("inf")
    x = x.to(dtype)
    p = kc.Pool(ssdv, 1, 1, D, 16, n)
    p.append([0], x.cuda(), x.cuda().flip(3).contiguous())
    rk, rv = p.read([0], n)
    x64 = x.double().numpy()
    np.testing.assert_array_equal(rk, kc.held(x64))
    np.testing.assert_array_equal(rv, kc.held(x64[..., ::-1].copy()))
    assert np.isnan(rk[0, 15, 0, :16]).all() and not np.isnan(rk[0, 15, 0, 16:]).any()
    assert rk[0, 15, 0, 20] == 1680 and rk[0, 15, 0, 40] == -1680


def test_every_bf16_maximum_and_tie(ssdv):
    """Every positive bf16 maximum from 2^-20 to 2048 with elements at k / 14 of it: scales and codes at their borders."""
    a = torch.arange(0x3580, 0x4500, dtype=torch.int32).to(torch.int16).view(BF16)
    frac = torch.tensor([1, 13 / 14, 11 / 14, 9 / 14, 0.5, 5 / 14, 3 / 14, 1 / 14, -1, -13 / 14, -6 / 7, -5 / 7, -0.25, -3 / 14,
                         -1 / 14, 0])
    x = (a.float()[:, None] * frac).to(BF16).float()
    pad = -x.shape[0] % 4
    x = torch.cat([x, torch.zeros(pad, 16)]).reshape(1, -1, 1, 64)
    for dtype in (BF16, F32):
        y = x.to(dtype)
        p = kc.Pool(ssdv, 1, 1, 64, 64, y.shape[1])
        p.append([0], y.cuda(), y.cuda())
        rk, rv = p.read([0], y.shape[1])
        want = kc.held(y.double().numpy())
        np.testing.assert_array_equal(rk, want)
        np.testing.assert_array_equal(rv, want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_other_tokens_keep_theirs(ssdv, D):
    """Ragged appends into partly filled blocks, zero counts among them, leave the tokens before them and all other
    requests alone; a rejected draft's place is written again."""
    B, H, page, T = 5, 2, 32, 200
    p = kc.Pool(ssdv, B, H, D, page, T, seed=3, fill=0xFF)
    want = np.zeros((2, B, T, H, D))
    lens = np.zeros(B, dtype=int)
    g = np.random.default_rng(9)
    for step in range(12):
        n = int(g.integers(1, 24))
        new = g.integers(0, n + 1, B)
        k, k64 = kc.rows((B, n, H, D), BF16, 100 + step)
        v, v64 = kc.rows((B, n, H, D), BF16, 200 + step)
        p.append(lens, k, v, n_new=new)
        for b in range(B):
            want[0, b, lens[b]:lens[b] + new[b]] = kc.held(k64[b, :new[b]])
            want[1, b, lens[b]:lens[b] + new[b]] = kc.held(v64[b, :new[b]])
        keep = np.minimum(new, g.integers(0, n + 1, B))  # the rest is rejected
        lens = np.minimum(lens + keep, T - 24)
    rk, rv = p.read(np.zeros(B), T, count=lens)
    for b in range(B):
        want[:, b, lens[b]:] = 0
    np.testing.assert_array_equal(rk, want[0])
    np.testing.assert_array_equal(rv, want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["fused", "heads_first", "offset", "repeated"])
def test_strides_and_alignment(ssdv, dtype, form):
    B, n, H, D = 2, 21, 4, 64
    x, x64 = kc.rows((B, n, 3, H, D), dtype, 4)
    if form == "fused":
        k, v, k64, v64 = x[:, :, 1], x[:, :, 2], x64[:, :, 1], x64[:, :, 2]
    elif form == "heads_first":
        y = x.permute(0, 3, 2, 1, 4).contiguous()  # [B, H, 3, n, D]
        k, v = y[:, :, 0].permute(0, 2, 1, 3), y[:, :, 1].permute(0, 2, 1, 3)
        k64, v64 = x64[:, :, 0], x64[:, :, 1]
    elif form == "offset":  # rows that start off a 16-byte boundary
        flat = torch.zeros(x.numel() + 1, dtype=dtype, device="cuda")
        flat[1:] = x.reshape(-1)
        y = flat[1:].view(x.shape)
        k, v, k64, v64 = y[:, :, 0], x[:, :, 1], x64[:, :, 0], x64[:, :, 1]
    else:  # one key for every head
        k, v = x[:, :, 0, :1].expand(B, n, H, D), x[:, :, 1]
        k64, v64 = np.broadcast_to(x64[:, :, 0, :1], (B, n, H, D)), x64[:, :, 1]
    p = kc.Pool(ssdv, B, H, D, 16, n + 3)
    p.append([3, 0], k, v)
    rk, rv = p.read([3, 0], n)
    np.testing.assert_array_equal(rk, kc.held(k64))
    np.testing.assert_array_equal(rv, kc.held(v64))


def test_errors_stay_with_their_request(ssdv):
    """Bad lengths, counts and pages: nothing is written for them, reads give NaN, the status names them, and the other
    requests are served."""
    B, n, H, D, page = 6, 20, 2, 128, 16
    p = kc.Pool(ssdv, B, H, D, page, 48)  # 3 pages a request
    k, k64 = kc.rows((B, n, H, D), BF16, 1)
    good = p.table.clone()
    before = p.cache.clone()
    p.table[1, 1] = -1
    p.table[2, 0] = p.cache.shape[0]
    lens = [0, 0, 0, -1, 29, 28]
    ws = ssdv.make_kv_workspace()
    p.append(lens, k, k, workspace=ws)
    assert ssdv.read_status(ws) == 12 and ssdv.read_status(ws) == 0
    p.append([0, 0, 0, -1, 29, 28], k, k, workspace=ws, n_new=[n, 0, 0, 1, n, n])
    assert ssdv.read_status(ws) == 13
    p.append([0] * B, k, k, workspace=ws, n_new=[n, 0, 0, 0, 21, -1])
    assert ssdv.read_status(ws) == 13
    for b, pages in ((1, [1, 2]), (2, [0]), (3, [0, 1, 2])):  # untouched
        for j in pages:
            at = int(good[b, j])
            assert torch.equal(p.cache[at], before[at])
    rk, _ = ssdv.kv_read(p.cache, p.table, kc.ints([0, 0, 0, -1, 29, 28]), n, F32, workspace=ws)
    assert ssdv.read_status(ws) == 12
    rk = rk.double().cpu().numpy()
    want = kc.held(k64)
    np.testing.assert_array_equal(rk[0], want[0])
    np.testing.assert_array_equal(rk[5], want[5])
    np.testing.assert_array_equal(rk[1, :16], want[1, :16])
    np.testing.assert_array_equal(rk[2, 16:], want[2, 16:])
    for bad in (rk[1, 16:], rk[2, :16], rk[3], rk[4]):
        assert np.isnan(bad).all()


def test_pool_past_32_bits(ssdv):
    """Pages whose bytes lie past 2^32, in a pool of 4.9 GB."""
    H, D, page = 8, 128, 128
    n_pages = (5 << 30) // ssdv.lib().ssd_kv_page_bytes(H, D, page) - 1
    cache = ssdv.make_kv_cache(n_pages, H, D, page, device="cuda")
    table = kc.ints([[n_pages - 1, 3, n_pages - 2]])
    k, k64 = kc.rows((1, 300, H, D), BF16, 8)
    v, v64 = kc.rows((1, 300, H, D), BF16, 9)
    ssdv.kv_append(cache, table, kc.ints([50]), k, v)
    rk, rv = ssdv.kv_read(cache, table, kc.ints([50]), 300, F32)
    np.testing.assert_array_equal(rk.double().cpu().numpy(), kc.held(k64))
    np.testing.assert_array_equal(rv.double().cpu().numpy(), kc.held(v64))
    assert int(cache[4:n_pages - 2].count_nonzero()) == 0


def test_empty_calls_and_streams(ssdv):
    p = kc.Pool(ssdv, 2, 2, 64, 16, 40)
    none = torch.empty(2, 0, 2, 64, dtype=BF16, device="cuda")
    p.append([0, 0], none, none)
    k, v = ssdv.kv_read(p.cache, p.table, kc.ints([0, 0]), 0)
    assert k.shape == (2, 0, 2, 64)
    x, x64 = kc.rows((2, 9, 2, 64), BF16, 3)
    side = torch.cuda.Stream()
    lens = kc.ints([0, 5])
    torch.cuda.synchronize()
    ssdv.kv_append(p.cache, p.table, lens, x, x, stream=side)
    rk, rv = ssdv.kv_read(p.cache, p.table, lens, 9, F32, stream=side)
    side.synchronize()
    np.testing.assert_array_equal(rk.double().cpu().numpy(), kc.held(x64))
    np.testing.assert_array_equal(rv.double().cpu().numpy(), kc.held(x64))
