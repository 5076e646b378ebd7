"""kv_plan and qk_norm_rope refuse bad arguments on the host, before any launch
(no GPU needed)."""
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


def test_plan_arguments(lib):
    names = ("table", "held", "free", "n_free", "B", "max_pages", "n_pages", "page", "len", "new", "n", "shared", "out_table",
             "out_held", "out_free", "out_n", "slots", "ws", "size")

    def plan(**kw):
        far = ctypes.c_void_p(1 << 20)
        args = dict(zip(names, (P, P, P, P, 4, 8, 64, 64, P, None, 5, None, far, far, far, far, P, P, 1 << 12)), **kw)
        return lib.ssd_kv_plan(*args.values(), None)

    for name in ("table", "held", "free", "n_free", "len", "out_table", "out_held", "out_free", "out_n", "ws"):
        assert plan(**{name: None}) == NULL, name
    for kw in (dict(B=0), dict(max_pages=0), dict(n_pages=0), dict(page=0), dict(page=24), dict(page=-16), dict(n=-1),
               dict(n=(1 << 30) + 1), dict(max_pages=1 << 20, page=1 << 11)):
        assert plan(**kw) == SHAPE, kw
    for name in ("table", "held", "free", "n_free", "len", "new", "shared", "out_table", "out_held", "out_free", "out_n"):
        assert plan(**{name: ODD}) == ALIGN, name
    assert plan(slots=ctypes.c_void_p(4100)) == ALIGN and plan(ws=ctypes.c_void_p(4104)) == ALIGN
    assert plan(size=256 + 16 * 5 - 1) == WORKSPACE and lib.ssd_kv_plan_workspace_bytes(4) == 256 + 16 * 5
    assert lib.ssd_kv_plan_workspace_bytes(0) == 0
    # an output that lies partly over its input, at either end
    for name, at in (("out_table", 4100), ("out_table", 4096 - 4 * 31), ("out_held", 4108), ("out_free", 4096 + 252)):
        assert plan(**{name: ctypes.c_void_p(at)}) == SHAPE, (name, at)


def test_rope_arguments(lib):
    neg, other = (ctypes.c_int64 * 3)(1024, -128, 128), (ctypes.c_int64 * 3)(1024, 256, 128)
    names = ("q", "qs", "k", "ks", "dt", "len", "new", "B", "n", "heads", "kv", "dim", "qw", "kw", "eps", "freq", "rot", "il",
             "oq", "oqs", "ok", "oks", "ws", "size")

    def rope(**kw):
        args = dict(zip(names, (P, ST, P, ST, 0, P, None, 2, 3, 8, 2, 128, P, P, 1e-6, P, 128, 0, P, ST, P, ST, P, 256)), **kw)
        return lib.ssd_qk_norm_rope(*args.values(), None)

    for name in ("q", "qs", "k", "ks", "len", "freq", "oq", "oqs", "ok", "oks", "ws"):
        assert rope(**{name: None}) == NULL, name
    for kw in (dict(B=0), dict(n=0), dict(n=(1 << 30) + 1), dict(heads=0), dict(heads=65536), dict(kv=-1), dict(kv=65536),
               dict(dim=96), dict(rot=8), dict(rot=-16), dict(rot=144), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(qs=neg), dict(ks=neg), dict(oqs=neg), dict(oks=neg), dict(B=1 << 20, n=1 << 20),
               dict(qs=other), dict(oks=other)):
        assert rope(**kw) == SHAPE, kw
    for name in ("q", "k", "len", "new", "qw", "kw", "freq", "oq", "ok", "ws"):
        assert rope(**{name: ODD}) == ALIGN, name
    assert rope(qw=ctypes.c_void_p(4100)) == ALIGN and rope(q=ctypes.c_void_p(4098), dt=1) == ALIGN
    assert rope(dt=2) == DTYPE and rope(size=255) == WORKSPACE


def test_binding_refuses():
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ssdv.kv_plan(ints(2, 4), ints(2), ints(9), ints(1), ints(2), 3, 16)
    for n, page in ((-1, 16), (1 << 31, 16), (3, (1 << 32) + 16), (3, 0), (3, -16)):
        with pytest.raises(ValueError, match="32-bit"):
            ssdv.kv_plan(ints(2, 4), ints(2), ints(9), ints(1), ints(2), n, page)
    with pytest.raises(ValueError, match="max_pages"):
        ssdv.kv_plan(ints(8), ints(2), ints(9), ints(1), ints(2), 3, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ssdv.qk_norm_rope(torch.zeros(2, 3, 8, 64), torch.zeros(2, 3, 2, 64), ints(2))
    with pytest.raises(ValueError, match="n_heads"):
        ssdv.qk_norm_rope(torch.zeros(2, 3, 64), None, ints(2))
    for n in (0, -1, 1 << 31):
        with pytest.raises(ValueError, match="pool"):
            ssdv.make_kv_pool(n, device="cpu")
    free, n_free = ssdv.make_kv_pool(3, device="cpu")
    assert free.tolist() == [2, 1, 0] and n_free.tolist() == [3]


def test_sinks_arguments(lib):
    c = ctypes.byref(ssdv.KvCacheStruct(pages=4096, n_pages=8, n_kv_heads=2, head_dim=128, page_size=64, max_pages=4,
                                        page_table=4096))

    def att(window, sinks):
        return lib.ssd_kv_attention_sinks(c, P, None, P, ST, 0, 2, 3, 8, 0.1, window, sinks, 0, P, None, P, 16, None)

    assert att(-1, 0) == SHAPE and att(0, -1) == SHAPE and att(64, -(1 << 31)) == SHAPE and att(64, 4) == WORKSPACE


def test_shared_arguments(lib):
    def cache(**kw):
        args = dict(pages=4096, n_pages=8, n_kv_heads=2, head_dim=128, page_size=64, max_pages=4, page_table=4096)
        args.update(kw)
        return ctypes.byref(ssdv.KvCacheStruct(**args))

    def att(c=None, lens=P, nq=None, q=P, qs=ST, dt=0, B=2, n=3, heads=8, scale=0.1, start=P, shared=P, G=2, out=P, lse=None,
            ws=P, size=1 << 40):
        return lib.ssd_kv_attention_shared(c or cache(), lens, nq, q, qs, dt, B, n, heads, scale, start, shared, G, 0, out, lse,
                                           ws, size, None)

    neg = (ctypes.c_int64 * 3)(-1024, 128, 128)
    for kw in (dict(lens=None), dict(q=None), dict(qs=None), dict(out=None), dict(ws=None), dict(start=None), dict(shared=None),
               dict(c=cache(pages=None)), dict(c=cache(page_table=None))):
        assert att(**kw) == NULL, kw
    for kw in (dict(B=0), dict(B=65536), dict(n=0), dict(n=33), dict(heads=7), dict(heads=512), dict(G=0), dict(G=65536),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=3e38), dict(qs=neg), dict(c=cache(head_dim=96)),
               dict(c=cache(page_size=24))):
        assert att(**kw) == SHAPE, kw
    for kw in (dict(lens=ODD), dict(nq=ODD), dict(q=ODD), dict(start=ODD), dict(shared=ODD), dict(out=ODD), dict(lse=ODD),
               dict(ws=ODD)):
        assert att(**kw) == ALIGN, kw
    need = lib.ssd_kv_shared_workspace_bytes(2, 3, 8, 2, 128, 2)
    assert need > 256 and att(size=need - 1) == WORKSPACE and att(dt=3) == DTYPE
    for bad in ((0, 3, 8, 2, 128, 2), (65536, 3, 8, 2, 128, 2), (2, 0, 8, 2, 128, 2), (2, 33, 8, 2, 128, 2), (2, 3, 7, 2, 128, 2),
                (2, 3, 8, 2, 96, 2), (2, 3, 8, 2, 128, 0), (2, 3, 8, 2, 128, 65536)):
        assert lib.ssd_kv_shared_workspace_bytes(*bad) == 0, bad
