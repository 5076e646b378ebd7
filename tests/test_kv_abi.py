"""The key/value cache calls refuse bad arguments on the host, before any
launch (no GPU needed), and the binding refuses what it cannot pass on."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_draft_gb300 import ssdv

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 9
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)
ST = (ctypes.c_int64 * 3)(1024, 128, 128)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_draft_gb300 import build
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    return ssdv._declare(ctypes.CDLL(build.build()))


def cache(**kw):
    args = dict(pages=4096, n_pages=8, n_kv_heads=2, head_dim=128, page_size=64, max_pages=4, page_table=4096)
    args.update(kw)
    return ctypes.byref(ssdv.KvCacheStruct(**args))


BAD_CACHES = [
    (dict(pages=None), NULL), (dict(page_table=None), NULL), (dict(pages=4104), ALIGN), (dict(page_table=4097), ALIGN),
    (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=-16), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(page_size=1 << 20, max_pages=1 << 11), SHAPE),
]


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches(lib, bad, code):
    c = cache(**bad)
    assert lib.ssd_kv_append(c, P, None, P, ST, P, ST, 0, 2, 3, P, 1 << 24, None) == code
    assert lib.ssd_kv_read(c, P, None, 0, 2, 3, P, P, P, 1 << 24, None) == code
    assert lib.ssd_kv_attention(c, P, None, P, ST, 0, 2, 3, 8, 0.1, 0, 0, P, None, P, 1 << 28, None) == code


def test_append_and_read_arguments(lib):
    neg = (ctypes.c_int64 * 3)(1024, -128, 128)

    def append(c=None, lens=P, news=None, k=P, ks=ST, v=P, vs=ST, dt=0, B=2, n=3, ws=P, size=1 << 10):
        return lib.ssd_kv_append(c or cache(), lens, news, k, ks, v, vs, dt, B, n, ws, size, None)

    def read(c=None, start=P, count=None, dt=0, B=2, n=3, k=P, v=P, ws=P, size=1 << 10):
        return lib.ssd_kv_read(c or cache(), start, count, dt, B, n, k, v, ws, size, None)

    assert lib.ssd_kv_append(None, P, None, P, ST, P, ST, 0, 2, 3, P, 1 << 10, None) == NULL
    for kw in (dict(lens=None), dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(ws=None)):
        assert append(**kw) == NULL, kw
    for kw in (dict(B=0), dict(n=0), dict(n=-1), dict(ks=neg), dict(vs=neg), dict(B=1 << 30, n=1 << 20)):
        assert append(**kw) == SHAPE, kw
    for kw in (dict(lens=ODD), dict(news=ODD), dict(k=ODD), dict(v=ODD), dict(ws=ODD), dict(k=ctypes.c_void_p(4098), dt=1)):
        assert append(**kw) == ALIGN, kw
    assert append(dt=2) == DTYPE and append(size=255) == WORKSPACE
    for kw in (dict(start=None), dict(k=None), dict(v=None), dict(ws=None)):
        assert read(**kw) == NULL, kw
    for kw in (dict(B=0), dict(n=0), dict(B=1 << 30, n=1 << 20)):
        assert read(**kw) == SHAPE, kw
    for kw in (dict(start=ODD), dict(count=ODD), dict(k=ctypes.c_void_p(4104)), dict(v=ctypes.c_void_p(4104))):
        assert read(**kw) == ALIGN, kw
    assert read(dt=-1) == DTYPE and read(size=0) == WORKSPACE


def test_attention_arguments(lib):
    def att(c=None, lens=P, nq=None, q=P, qs=ST, dt=0, B=2, n=3, heads=8, scale=0.1, window=0, out=P, lse=None, ws=P,
            size=1 << 30):
        return lib.ssd_kv_attention(c or cache(), lens, nq, q, qs, dt, B, n, heads, scale, window, 0, out, lse, ws, size,
                                    None)

    for kw in (dict(lens=None), dict(q=None), dict(qs=None), dict(out=None), dict(ws=None)):
        assert att(**kw) == NULL, kw
    for kw in (dict(B=0), dict(B=65536), dict(n=0), dict(n=33), dict(heads=0), dict(heads=7), dict(heads=1),
               dict(heads=2 * 129), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert att(**kw) == SHAPE, kw
    for kw in (dict(lens=ODD), dict(nq=ODD), dict(q=ODD), dict(out=ctypes.c_void_p(4104)), dict(lse=ODD), dict(ws=ODD)):
        assert att(**kw) == ALIGN, kw
    assert att(dt=5) == DTYPE
    need = lib.ssd_kv_workspace_bytes(3, 8, 2, 128)
    assert need >= 256 and att(size=need - 1) == WORKSPACE


def test_sizes(lib):
    assert lib.ssd_kv_page_bytes(2, 128, 64) == 2 * 64 * (2 * 64 + 2 * 8)  # 4.5 bits an element, twice
    for bad in ((0, 128, 64), (2, 80, 64), (2, 128, 0), (2, 128, 40)):
        assert lib.ssd_kv_page_bytes(*bad) == 0
    assert lib.ssd_kv_workspace_bytes(0, 0, 0, 0) == 256
    for bad in ((33, 8, 2, 128), (-1, 8, 2, 128), (1, 8, 3, 128), (1, 2, 8, 128), (1, 8, 0, 128), (1, 8, 2, 100)):
        assert lib.ssd_kv_workspace_bytes(*bad) == 0
    for code in (12, 13):
        assert lib.ssd_status_str(code).decode().startswith(ssdv.STATUS_NAMES[code])


def test_binding_refuses_host_tensors_and_shapes(lib, monkeypatch):
    monkeypatch.setattr(ssdv, "_lib", lib)
    with pytest.raises(ValueError, match="head_dim"):
        ssdv.make_kv_cache(4, 2, 80)
    with pytest.raises(ValueError, match="page_size"):
        ssdv.make_kv_cache(4, 2, 64, page_size=20)
    with pytest.raises(ValueError, match="n_pages"):
        ssdv.make_kv_cache(0, 2, 64)
    with pytest.raises(ValueError, match="no workspace"):
        ssdv.make_kv_workspace(40, 8, 2, 128)
    c = torch.zeros(4, 2, 4, 18 * 64, dtype=torch.uint8)
    t = torch.zeros(2, 4, dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: ssdv.kv_append(c, t, n, x, x), lambda: ssdv.kv_read(c, t, n, 3),
                 lambda: ssdv.kv_attention(c, t, n, x)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
