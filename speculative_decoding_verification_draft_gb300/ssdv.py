"""Thin ctypes binding of libssdv (C ABI in ``include/ssdv.h``).

Argument marshalling only: every function checks tensor dtypes, shapes and
devices, passes raw device pointers and the current CUDA stream to the
library, and turns a non-zero status into ``SsdError``.  All computation runs
in the library's CUDA kernels; there is no CPU fallback.  If ``libssdv.so`` is
missing the first call raises -- build it with ``build.build()`` (or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
import threading
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libssdv.so")

SSD_BF16, SSD_F32 = 0, 1
NSTAT_VERIFY = 10
NSTAT_SAGUARO = 10
MAX_TOPK = 8

STATUS_NAMES = {
    0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_DTYPE", 4: "SSD_ERR_ALIGN",
    5: "SSD_ERR_TOKEN_RANGE", 6: "SSD_ERR_TEMPERATURE", 7: "SSD_ERR_CUDA", 8: "SSD_ERR_UNSUPPORTED",
    9: "SSD_ERR_WORKSPACE", 10: "SSD_ERR_GAMMA", 11: "SSD_ERR_DRAW", 12: "SSD_ERR_PAGE", 13: "SSD_ERR_LENGTH",
}


class SsdError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {detail}")


_lock = threading.Lock()
_lib = None


class KvCacheStruct(ctypes.Structure):
    """ssd_kv_cache of include/ssdv.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("page_table", ctypes.c_void_p)]


def _declare(lib):
    P, I, U64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float, ctypes.c_size_t
    lib.ssd_workspace_bytes.argtypes = [I, I]
    lib.ssd_workspace_bytes.restype = SZ
    lib.ssd_workspace_init.argtypes = [P, SZ, P]
    lib.ssd_verify.argtypes = [P, P, I, P, I, I, I, F, U64, P, P, P, SZ, P]
    lib.ssd_verify_ragged.argtypes = [P, P, I, P, I, I, I, P, P, U64, P, P, P, SZ, P]
    lib.ssd_verify_ragged_pipelined.argtypes = [P, P, I, P, I, I, I, P, P, U64, P, P, P, SZ, P]
    lib.ssd_verify_noalloc.argtypes = [P, P, I, P, I, I, I, F, U64, P, P, P]
    lib.ssd_verify_pipelined.argtypes = [P, P, I, P, I, I, I, F, U64, P, P, P, SZ, P]
    lib.ssd_saguaro_prespec.argtypes = [P, P, I, I, I, I, I, I, F, U64, P, P, P, SZ, P]
    lib.ssd_saguaro_workspace_bytes.argtypes = [I, I, I]
    lib.ssd_saguaro_workspace_bytes.restype = SZ
    lib.ssd_debug_rowstats.argtypes = [P, P, I, P, I, I, I, F, U64, P, P, P, P, SZ, P]
    lib.ssd_debug_saguaro_stats.argtypes = [P, P, I, I, I, I, I, I, F, U64, P, P, P, P, SZ, P]
    lib.ssd_verify_saguaro.argtypes = [P, P, I, P, I, I, I, I, I, F, U64, P, P, P, P, P, P, P, SZ, P]
    lib.ssd_cache_check.argtypes = [P, P, P, I, I, I, P, P, P]
    lib.ssd_verify_saguaro_draft.argtypes = [P, P, I, P, I, I, I, F, U64, P, P, P, SZ, P]
    lib.ssd_verify_top_p.argtypes = [P, P, I, P, I, I, I, F, F, U64, P, P, P, SZ, P]
    lib.ssd_verify_top_p_workspace_bytes.argtypes = [I, I]
    lib.ssd_verify_top_p_workspace_bytes.restype = SZ
    lib.ssd_kv_page_bytes.argtypes = [I, I, I]
    lib.ssd_kv_page_bytes.restype = SZ
    lib.ssd_kv_workspace_bytes.argtypes = [I, I, I, I]
    lib.ssd_kv_workspace_bytes.restype = SZ
    lib.ssd_kv_append.argtypes = [P, P, P, P, P, P, P, I, I, I, P, SZ, P]
    lib.ssd_kv_read.argtypes = [P, P, P, I, I, I, P, P, P, SZ, P]
    lib.ssd_kv_attention.argtypes = [P, P, P, P, P, I, I, I, I, F, I, I, P, P, P, SZ, P]
    lib.ssd_read_status.argtypes = [P, SZ, P, P]
    lib.ssd_stream_capture_id.argtypes = [P, P]
    lib.ssd_debug_uniforms.argtypes = [U64, I, I, P, P]
    lib.ssd_status_str.argtypes = [I]
    lib.ssd_status_str.restype = ctypes.c_char_p
    lib.ssd_last_error.argtypes = []
    lib.ssd_last_error.restype = ctypes.c_char_p
    for name in ("ssd_workspace_init", "ssd_verify", "ssd_verify_noalloc", "ssd_verify_pipelined",
                 "ssd_verify_ragged", "ssd_verify_ragged_pipelined", "ssd_saguaro_prespec", "ssd_debug_rowstats",
                 "ssd_debug_saguaro_stats", "ssd_read_status",
                 "ssd_verify_saguaro", "ssd_cache_check", "ssd_verify_saguaro_draft", "ssd_verify_top_p",
                 "ssd_kv_append", "ssd_kv_read", "ssd_kv_attention", "ssd_stream_capture_id", "ssd_debug_uniforms"):
        getattr(lib, name).restype = I
    return lib


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY):
                raise RuntimeError(f"{LIBRARY} is missing: build the CUDA library first "
                                   "(speculative_decoding_verification_draft_gb300.build.build())")
            _lib = _declare(ctypes.CDLL(LIBRARY))
    return _lib


def _check(status: int):
    if status != 0:
        raise SsdError(status, lib().ssd_last_error().decode())


def _dtype_code(t: torch.Tensor, name: str = "logits") -> int:
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    if t.dtype == torch.float32:
        return SSD_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


TOPK_SOURCES = {"residual": 0, "draft": 1}


def _source(source: str) -> int:
    if source not in TOPK_SOURCES:
        raise ValueError(f"top-k source must be one of {sorted(TOPK_SOURCES)}, got {source!r}")
    return TOPK_SOURCES[source]


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_ws_cache = {}


def workspace_bytes(B: int, gamma_max: int) -> int:
    return int(lib().ssd_workspace_bytes(B, gamma_max))


def make_workspace(B: int, gamma_max: int, device=None) -> torch.Tensor:
    """A zeroed device workspace for batches of up to B requests / gamma_max."""
    n = workspace_bytes(B, gamma_max)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _ws_key(device):
    device = torch.device(device if device is not None else "cuda")
    index = device.index if device.index is not None else torch.cuda.current_device()
    return (index, torch.cuda.current_stream(index).cuda_stream)


def _workspace(B: int, gmax: int, device, given: Optional[torch.Tensor]):
    if given is not None:
        return given
    key = _ws_key(device)
    need = workspace_bytes(B, gmax)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


_sag_ws_cache = {}


def saguaro_workspace_bytes(B: int, gamma: int, V: int) -> int:
    return int(lib().ssd_saguaro_workspace_bytes(B, gamma, V))


def make_saguaro_workspace(B: int, gamma: int, V: int, device=None) -> torch.Tensor:
    """A zeroed device workspace for Saguaro calls of up to B requests, gamma, V."""
    n = saguaro_workspace_bytes(B, gamma, V)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _saguaro_workspace(B: int, g: int, V: int, device, given: Optional[torch.Tensor]):
    # kept apart from the verification workspaces: a pipelined verification
    # call may write its workspace while the previous kernel still runs
    if given is not None:
        return given
    key = _ws_key(device)
    need = saguaro_workspace_bytes(B, g, V)
    ws = _sag_ws_cache.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=device)
        _sag_ws_cache[key] = ws
    return ws


def verify(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
           temperature: float, seed: int, out_tokens: Optional[torch.Tensor] = None,
           n_accepted: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           stream=None):
    """ssd_verify: target [B, g+1, V], draft [B, g, V], draft_tokens [B, g] int32.

    Returns (out_tokens [B, g+1] int32, n_accepted [B] int32)."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(B, g, dev, workspace)
    dptr = _dev(draft, "draft_logits", target.dtype) if draft is not None else None
    if draft is not None and tuple(draft.shape) != (B, g, V):
        raise ValueError("draft_logits must be [B, gamma, V]")
    if tuple(draft_tokens.shape) != (B, g):
        raise ValueError("draft_tokens must be [B, gamma]")
    _check(lib().ssd_verify(_dev(target, "target_logits"), dptr, _dtype_code(target),
                            _dev(draft_tokens, "draft_tokens", torch.int32), B, g, V, float(temperature),
                            int(seed) & ((1 << 64) - 1), _dev(out_tokens, "out_tokens", torch.int32),
                            _dev(n_accepted, "n_accepted", torch.int32), _dev(ws, "workspace"),
                            ws.numel(), _stream(stream)))
    return out_tokens, n_accepted


def verify_pipelined(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                     temperature: float, seed: int, out_tokens: Optional[torch.Tensor] = None,
                     n_accepted: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None):
    """ssd_verify_pipelined: ssd_verify for a chain of calls whose inputs were
    complete before the previous verification call on the stream completed."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(B, g, dev, workspace)
    dptr = _dev(draft, "draft_logits", target.dtype) if draft is not None else None
    if draft is not None and tuple(draft.shape) != (B, g, V):
        raise ValueError("draft_logits must be [B, gamma, V]")
    if tuple(draft_tokens.shape) != (B, g):
        raise ValueError("draft_tokens must be [B, gamma]")
    _check(lib().ssd_verify_pipelined(_dev(target, "target_logits"), dptr, _dtype_code(target),
                                      _dev(draft_tokens, "draft_tokens", torch.int32), B, g, V, float(temperature),
                                      int(seed) & ((1 << 64) - 1), _dev(out_tokens, "out_tokens", torch.int32),
                                      _dev(n_accepted, "n_accepted", torch.int32), _dev(ws, "workspace"),
                                      ws.numel(), _stream(stream)))
    return out_tokens, n_accepted


def verify_noalloc(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                   temperature: float, seed: int, out_tokens: torch.Tensor, n_accepted: torch.Tensor,
                   stream=None):
    """ssd_verify_noalloc: ssd_verify on the library's fixed device scratch.

    The caller passes the outputs (out_tokens [B, g+1], n_accepted [B] int32),
    so neither this wrapper nor the library allocates device memory."""
    B, W, V = target.shape
    g = W - 1
    dptr = _dev(draft, "draft_logits", target.dtype) if draft is not None else None
    if draft is not None and tuple(draft.shape) != (B, g, V):
        raise ValueError("draft_logits must be [B, gamma, V]")
    if tuple(draft_tokens.shape) != (B, g):
        raise ValueError("draft_tokens must be [B, gamma]")
    if tuple(out_tokens.shape) != (B, W) or tuple(n_accepted.shape) != (B,):
        raise ValueError("out_tokens must be [B, gamma+1] and n_accepted [B]")
    _check(lib().ssd_verify_noalloc(_dev(target, "target_logits"), dptr, _dtype_code(target),
                                    _dev(draft_tokens, "draft_tokens", torch.int32), B, g, V, float(temperature),
                                    int(seed) & ((1 << 64) - 1), _dev(out_tokens, "out_tokens", torch.int32),
                                    _dev(n_accepted, "n_accepted", torch.int32), _stream(stream)))
    return out_tokens, n_accepted


def verify_ragged(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor,
                  gamma: torch.Tensor, temperature: torch.Tensor, seed: int,
                  out_tokens: Optional[torch.Tensor] = None, n_accepted: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None, pipelined: bool = False):
    """ssd_verify_ragged: per-request gamma [B] int32 and temperature [B] float32.

    pipelined=True calls ssd_verify_ragged_pipelined: the inputs must have been
    complete before the previous verification call on the stream completed."""
    B, W, V = target.shape
    gmax = W - 1
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(B, gmax, dev, workspace)
    fn = lib().ssd_verify_ragged_pipelined if pipelined else lib().ssd_verify_ragged
    _check(fn(_dev(target, "target_logits"), _dev(draft, "draft_logits", target.dtype), _dtype_code(target),
              _dev(draft_tokens, "draft_tokens", torch.int32), B, gmax, V, _dev(gamma, "gamma", torch.int32),
              _dev(temperature, "temperature", torch.float32), int(seed) & ((1 << 64) - 1),
              _dev(out_tokens, "out_tokens", torch.int32), _dev(n_accepted, "n_accepted", torch.int32),
              _dev(ws, "workspace"), ws.numel(), _stream(stream)))
    return out_tokens, n_accepted


def saguaro_prespec(target: torch.Tensor, draft: torch.Tensor, k: int, temperature: float, seed: int,
                    bonus_topk: Optional[torch.Tensor] = None, saguaro_tokens: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None, source: str = "residual"):
    """ssd_saguaro_prespec: returns (bonus_topk [B, g+1, k], saguaro_tokens [B, g+1]).
    source: "residual" (top-k of r_j) or "draft" (the draft's k largest logits)."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    if bonus_topk is None:
        bonus_topk = torch.empty(B, W, k, dtype=torch.int32, device=dev)
    if saguaro_tokens is None:
        saguaro_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    dptr = _dev(draft, "draft_logits", target.dtype) if g > 0 else None
    ws = _saguaro_workspace(B, g, V, dev, workspace)
    _check(lib().ssd_saguaro_prespec(_dev(target, "target_logits"), dptr, _dtype_code(target), B, g, V, int(k),
                                     _source(source), float(temperature), int(seed) & ((1 << 64) - 1),
                                     _dev(bonus_topk, "bonus_topk", torch.int32),
                                     _dev(saguaro_tokens, "saguaro_tokens", torch.int32), _dev(ws, "workspace"),
                                     ws.numel(), _stream(stream)))
    return bonus_topk, saguaro_tokens


def verify_saguaro(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor, k: int,
                   temperature: float, seed: int, workspace: Optional[torch.Tensor] = None, check: bool = True,
                   stream=None, source: str = "residual"):
    """ssd_verify_saguaro: one call for both; returns (out_tokens [B, g+1], n_accepted [B],
    bonus_topk [B, g+1, k], saguaro_tokens [B, g+1], hit [B] or None, n_hits [1] or None)."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    bonus_topk = torch.empty(B, W, k, dtype=torch.int32, device=dev)
    saguaro_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    hit = torch.empty(B, dtype=torch.int32, device=dev) if check else None
    n_hits = torch.empty(1, dtype=torch.int32, device=dev) if check else None
    ws = _saguaro_workspace(B, g, V, dev, workspace)
    dptr = _dev(draft, "draft_logits", target.dtype) if g > 0 else None
    tptr = _dev(draft_tokens, "draft_tokens", torch.int32) if g > 0 else None
    _check(lib().ssd_verify_saguaro(_dev(target, "target_logits"), dptr, _dtype_code(target), tptr, B, g, V, int(k),
                                    _source(source), float(temperature), int(seed) & ((1 << 64) - 1), _dev(out_tokens, "out_tokens"),
                                    _dev(n_accepted, "n_accepted"), _dev(bonus_topk, "bonus_topk"),
                                    _dev(saguaro_tokens, "saguaro_tokens"),
                                    _dev(hit, "hit") if check else None, _dev(n_hits, "n_hits") if check else None,
                                    _dev(ws, "workspace"), ws.numel(), _stream(stream)))
    return out_tokens, n_accepted, bonus_topk, saguaro_tokens, hit, n_hits


_topp_ws_cache = {}


def verify_top_p(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor, temperature: float,
                 top_p: float, seed: int, out_tokens: Optional[torch.Tensor] = None,
                 n_accepted: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """ssd_verify_top_p: both distributions truncated to their top-p nuclei.
    Returns (out_tokens [B, g+1], n_accepted [B])."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    ws = workspace
    if ws is None:
        key = _ws_key(dev)
        need = int(lib().ssd_verify_top_p_workspace_bytes(B, g))
        ws = _topp_ws_cache.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=dev)
            _topp_ws_cache[key] = ws
    dptr = _dev(draft, "draft_logits", target.dtype) if draft is not None else None
    tptr = _dev(draft_tokens, "draft_tokens", torch.int32) if g > 0 else None
    _check(lib().ssd_verify_top_p(_dev(target, "target_logits"), dptr, _dtype_code(target), tptr, B, g, V,
                                  float(temperature), float(top_p), int(seed) & ((1 << 64) - 1),
                                  _dev(out_tokens, "out_tokens", torch.int32),
                                  _dev(n_accepted, "n_accepted", torch.int32), _dev(ws, "workspace"), ws.numel(),
                                  _stream(stream)))
    return out_tokens, n_accepted


def verify_saguaro_draft(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor, temperature: float,
                         seed: int, out_tokens: Optional[torch.Tensor] = None,
                         n_accepted: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         stream=None):
    """ssd_verify_saguaro_draft: draft tokens sampled from each position's Saguaro
    distribution.  Returns (out_tokens [B, g+1], n_accepted [B])."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _saguaro_workspace(B, g, V, dev, workspace)
    dptr = _dev(draft, "draft_logits", target.dtype) if g > 0 else None
    tptr = _dev(draft_tokens, "draft_tokens", torch.int32) if g > 0 else None
    _check(lib().ssd_verify_saguaro_draft(_dev(target, "target_logits"), dptr, _dtype_code(target), tptr, B, g, V,
                                          float(temperature), int(seed) & ((1 << 64) - 1),
                                          _dev(out_tokens, "out_tokens", torch.int32),
                                          _dev(n_accepted, "n_accepted", torch.int32), _dev(ws, "workspace"),
                                          ws.numel(), _stream(stream)))
    return out_tokens, n_accepted


def cache_check(bonus_topk: torch.Tensor, out_tokens: torch.Tensor, n_accepted: torch.Tensor, stream=None):
    """ssd_cache_check: (hit [B], n_hits [1])."""
    B, W, k = bonus_topk.shape
    dev = bonus_topk.device
    hit = torch.empty(B, dtype=torch.int32, device=dev)
    n_hits = torch.empty(1, dtype=torch.int32, device=dev)
    _check(lib().ssd_cache_check(_dev(bonus_topk, "bonus_topk", torch.int32), _dev(out_tokens, "out_tokens", torch.int32),
                                 _dev(n_accepted, "n_accepted", torch.int32), B, W - 1, k, _dev(hit, "hit"),
                                 _dev(n_hits, "n_hits"), _stream(stream)))
    return hit, n_hits


KV_BLOCK = 16  # tokens per block of a cache page, elements per scale
_KV_STATUS = 16  # bytes of a workspace that hold the status word
_kv_ws_cache = {}  # (device, stream): 0 and the stream's workspace
_kv_graph_ws = {}  # (device, stream): the last capture and its workspace
_HERE = contextlib.nullcontext()
# Small calls take a few microseconds on the GPU, so the binding of the cache calls
# packs its structures itself and asks torch as little as it can.
_KV_CACHE = struct.Struct("PqiiiiP")  # KvCacheStruct
_KV_STRIDES = struct.Struct("qqq")


@functools.lru_cache(maxsize=None)
def kv_workspace_bytes(n_q: int = 0, n_heads: int = 0, n_kv_heads: int = 0, head_dim: int = 0) -> int:
    return int(lib().ssd_kv_workspace_bytes(n_q, n_heads, n_kv_heads, head_dim))


def make_kv_workspace(n_q: int = 0, n_heads: int = 0, n_kv_heads: int = 0, head_dim: int = 0, device=None) -> torch.Tensor:
    """A zeroed device workspace for kv_append and kv_read (no arguments) or for
    kv_attention of up to n_q query tokens."""
    n = kv_workspace_bytes(n_q, n_heads, n_kv_heads, head_dim)
    if n == 0:
        raise ValueError(f"no workspace for n_q={n_q} n_heads={n_heads} n_kv_heads={n_kv_heads} head_dim={head_dim}")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def make_kv_cache(n_pages: int, n_kv_heads: int, head_dim: int, page_size: int = 64, device=None) -> torch.Tensor:
    """A pool of cache pages: uint8 [n_pages, n_kv_heads, page_size / 16, 18 * head_dim], all values zero."""
    if n_pages < 1 or lib().ssd_kv_page_bytes(n_kv_heads, head_dim, page_size) == 0:
        raise ValueError(f"no cache of n_pages={n_pages} n_kv_heads={n_kv_heads} head_dim={head_dim} "
                         f"page_size={page_size}: head_dim is 64, 128 or 256, page_size a multiple of {KV_BLOCK}")
    return torch.zeros(n_pages, n_kv_heads, page_size // KV_BLOCK, 18 * head_dim, dtype=torch.uint8,
                       device=device or "cuda")


def _kv_dev(t: torch.Tensor, name: str, dtype, index: int) -> int:
    """_dev of a tensor that has to be on the cache's device."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index or not t.is_contiguous():
        _dev(t, name)
        raise ValueError(f"{name} must live on the cache's device, cuda:{index}, not on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _kv_cache(cache: torch.Tensor, page_table: torch.Tensor, B: int):
    """(packed ssd_kv_cache, n_kv_heads, head_dim)"""
    ptr = _dev(cache, "cache", torch.uint8)
    table = _kv_dev(page_table, "page_table", torch.int32, cache.get_device())
    shape, width = cache.shape, page_table.shape
    if len(shape) != 4 or shape[3] % 18:
        raise ValueError("cache must be [n_pages, n_kv_heads, page_size / 16, 18 * head_dim] (make_kv_cache)")
    if len(width) != 2 or width[0] != B:
        raise ValueError(f"page_table must be [{B}, max_pages], got {list(width)}")
    n_pages, heads, blocks, block = shape
    dim = block // 18
    return _KV_CACHE.pack(ptr, n_pages, heads, dim, blocks * KV_BLOCK, width[1], table), heads, dim


def _kv_counts(t: Optional[torch.Tensor], name: str, B: int, index: int):
    if t is None:
        return None
    if t.shape != (B,):
        raise ValueError(f"{name} must be [{B}], got {list(t.shape)}")
    return _kv_dev(t, name, torch.int32, index)


def _kv_rows(t: torch.Tensor, name: str, heads: Optional[int], dim: int, index: int):
    """Pointer and packed strides of [B, n, heads, head_dim] rows: any strides but the last."""
    if t.get_device() != index:
        if not t.is_cuda:
            raise ValueError(f"{name} must live on a CUDA device")
        raise ValueError(f"{name} must live on the cache's device, cuda:{index}, not on {t.device}")
    shape, st = t.shape, t.stride()
    if len(shape) != 4 or shape[3] != dim or (heads is not None and shape[2] != heads):
        raise ValueError(f"{name} must be [B, n, {heads or 'n_heads'}, {dim}], got {list(shape)}")
    if st[3] != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return t.data_ptr(), _KV_STRIDES.pack(st[0], st[1], st[2])


def _kv_stream(stream, device):
    """(raw stream, context that makes it current, or None): outputs and workspaces are
    allocated on the stream that uses them.  The launch goes to the current device."""
    index = device.index
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"the cache is on {device}, which is not the current device")
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        return current, None
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"the cache is on {device}, the stream on {stream.device}")
    raw = _stream(stream)
    if raw == current:
        return raw, None
    return raw, torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                                  else torch.cuda.ExternalStream(raw, device=device))


def _capture_id(raw: int) -> int:
    """The number of the capture that a stream is in, 0 if it is in none."""
    n = ctypes.c_uint64(0)
    _check(lib().ssd_stream_capture_id(raw, ctypes.byref(n)))
    return n.value


def _kv_workspace(need: int, device, raw: int):
    """The stream's own workspace (called with the stream current).  The calls of a
    capture share one of their own, which the graph keeps: the stream's may be
    replaced by a larger one, and a graph may run beside the stream."""
    if need == 0:
        return torch.empty(16, dtype=torch.uint8, device=device)  # the call names the bad argument
    capture = _capture_id(raw) if torch._C._cuda_isCurrentStreamCapturing() else 0
    cache = _kv_graph_ws if capture else _kv_ws_cache
    of, ws = cache.get((device.index, raw), (0, None))
    if of != capture:
        ws = None
    if ws is None or ws.numel() < need:
        old, ws = ws, torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=device)
        # of a workspace only the status word is read before it is written
        if old is None:
            ws[:_KV_STATUS].zero_()
        else:
            ws[:_KV_STATUS].copy_(old[:_KV_STATUS])  # errors that nobody has read yet
        cache[(device.index, raw)] = (capture, ws)
    return ws


def kv_workspace(device=None, stream=None) -> Optional[torch.Tensor]:
    """The workspace that the kv_ calls without one use on this stream (None before
    the first), for read_status.  Inside a capture it is the one of the calls
    captured so far: kept, it tells the errors of the graph's last replay."""
    device = torch.device(device if device is not None else "cuda")
    index = device.index if device.index is not None else torch.cuda.current_device()
    raw = _stream(stream)
    capture = _capture_id(raw)
    of, ws = (_kv_graph_ws if capture else _kv_ws_cache).get((index, raw), (0, None))
    return ws if of == capture else None


def kv_append(cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              n_new: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """ssd_kv_append: write k, v [B, n, n_kv_heads, head_dim] (bf16 or fp32, any strides but the last) at positions
    kv_len[b] .. kv_len[b] + n_new[b] - 1.  kv_len is not changed."""
    B, n = k.shape[:2]
    c, heads, dim = _kv_cache(cache, page_table, B)
    index = cache.get_device()
    kp, ks = _kv_rows(k, "k", heads, dim, index)
    vp, vs = _kv_rows(v, "v", heads, dim, index)
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must have one shape and dtype")
    lens, news = _kv_counts(kv_len, "kv_len", B, index), _kv_counts(n_new, "n_new", B, index)
    if B == 0 or n == 0:
        return
    raw, ctx = _kv_stream(stream, cache.device)
    ws = workspace
    if ws is None:
        with ctx or _HERE:
            ws = _kv_workspace(256, cache.device, raw)
    _check(lib().ssd_kv_append(c, lens, news, kp, ks, vp, vs, _dtype_code(k, "k and v"), B, n,
                               _kv_dev(ws, "workspace", None, index), ws.numel(), raw))


def kv_read(cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor, n: int, dtype=torch.bfloat16,
            count: Optional[torch.Tensor] = None, out=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """ssd_kv_read: (k, v) [B, n, n_kv_heads, head_dim], the values held for positions start[b] .. start[b] +
    count[b] - 1 (rows past count[b] are zero); out: a pair of tensors to write them to."""
    B = page_table.shape[0]
    c, heads, dim = _kv_cache(cache, page_table, B)
    shape, device, index = (B, int(n), heads, dim), cache.device, cache.get_device()
    starts, counts = _kv_counts(start, "start", B, index), _kv_counts(count, "count", B, index)
    raw, ctx = _kv_stream(stream, device)
    ws = workspace
    with ctx or _HERE:
        k, v = out if out is not None else (torch.empty(shape, dtype=dtype, device=device),
                                            torch.empty(shape, dtype=dtype, device=device))
        if ws is None:
            ws = _kv_workspace(256, device, raw)
    if k.shape != shape or v.shape != shape or k.dtype != v.dtype:
        raise ValueError(f"out must be two tensors {list(shape)} of one dtype")
    if B == 0 or n == 0:
        return k, v
    _check(lib().ssd_kv_read(c, starts, counts, _dtype_code(k, "outputs"), B, int(n), _kv_dev(k, "out k", None, index),
                             _kv_dev(v, "out v", None, index), _kv_dev(ws, "workspace", None, index), ws.numel(), raw))
    return k, v


def kv_attention(cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, q: torch.Tensor,
                 n_q: Optional[torch.Tensor] = None, scale: Optional[float] = None, window: int = 0,
                 past_only: bool = False, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """ssd_kv_attention: q [B, n, n_heads, head_dim] (bf16 or fp32, any strides but the last), query i of request b at
    position kv_len[b] + i.  scale defaults to head_dim ** -0.5.  Returns out like q, contiguous, or (out, lse
    [B, n, n_heads] float32) with return_lse (or a given lse)."""
    shape, device = q.shape, cache.device
    B, n, heads = shape[:3]
    window = int(window)
    if not -1 << 31 <= window < 1 << 31:
        raise ValueError(f"window={window} is no 32-bit number")
    c, kv_heads, dim = _kv_cache(cache, page_table, B)
    index = cache.get_device()
    qp, qs = _kv_rows(q, "q", None, dim, index)
    lens, counts = _kv_counts(kv_len, "kv_len", B, index), _kv_counts(n_q, "n_q", B, index)
    raw, ctx = _kv_stream(stream, device)
    ws = workspace
    with ctx or _HERE:
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=device)
        if lse is None and return_lse:
            lse = torch.empty((B, n, heads), dtype=torch.float32, device=device)
        if ws is None and B and n:
            ws = _kv_workspace(kv_workspace_bytes(n, heads, kv_heads, dim), device, raw)
    if out.shape != shape or (lse is not None and lse.shape != (B, n, heads)):
        raise ValueError("out must be shaped like q and lse [B, n, n_heads]")
    if B and n:
        _check(lib().ssd_kv_attention(c, lens, counts, qp, qs, _dtype_code(q, "q"), B, n, heads,
                                      float(scale) if scale is not None else dim ** -0.5, window, int(past_only),
                                      _kv_dev(out, "out", q.dtype, index),
                                      _kv_dev(lse, "lse", torch.float32, index) if lse is not None else None,
                                      _kv_dev(ws, "workspace", None, index), ws.numel(), raw))
    return (out, lse) if lse is not None else out


def debug_rowstats(target, draft, draft_tokens, temperature, seed, workspace=None, stream=None):
    """ssd_debug_rowstats: (out_tokens, n_accepted, stats [B, g+1, 10] float32)."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    out_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    stats = torch.empty(B, W, NSTAT_VERIFY, dtype=torch.float32, device=dev)
    ws = _workspace(B, g, dev, workspace)
    dptr = _dev(draft, "draft_logits", target.dtype) if draft is not None else None
    _check(lib().ssd_debug_rowstats(_dev(target, "target_logits"), dptr, _dtype_code(target),
                                    _dev(draft_tokens, "draft_tokens", torch.int32), B, g, V, float(temperature),
                                    int(seed) & ((1 << 64) - 1), _dev(out_tokens, "out_tokens"),
                                    _dev(n_accepted, "n_accepted"), _dev(stats, "stats"), _dev(ws, "workspace"),
                                    ws.numel(), _stream(stream)))
    return out_tokens, n_accepted, stats


def debug_saguaro_stats(target, draft, k, temperature, seed, workspace=None, stream=None, source="residual"):
    """ssd_debug_saguaro_stats: (bonus_topk, saguaro_tokens, stats [B, g+1, 10])."""
    B, W, V = target.shape
    g = W - 1
    dev = target.device
    bonus_topk = torch.empty(B, W, k, dtype=torch.int32, device=dev)
    saguaro_tokens = torch.empty(B, W, dtype=torch.int32, device=dev)
    stats = torch.empty(B, W, NSTAT_SAGUARO, dtype=torch.float32, device=dev)
    dptr = _dev(draft, "draft_logits", target.dtype) if g > 0 else None
    ws = _saguaro_workspace(B, g, V, dev, workspace)
    _check(lib().ssd_debug_saguaro_stats(_dev(target, "target_logits"), dptr, _dtype_code(target), B, g, V,
                                         int(k), _source(source), float(temperature), int(seed) & ((1 << 64) - 1),
                                         _dev(bonus_topk, "bonus_topk"), _dev(saguaro_tokens, "saguaro_tokens"),
                                         _dev(stats, "stats"), _dev(ws, "workspace"), ws.numel(),
                                         _stream(stream)))
    return bonus_topk, saguaro_tokens, stats


def debug_uniforms(seed: int, B: int, W: int, device=None, stream=None) -> torch.Tensor:
    """ssd_debug_uniforms: [B, W, 3] float32 (accept, resample, Saguaro draws)."""
    out = torch.empty(B, W, 3, dtype=torch.float32, device=device or "cuda")
    _check(lib().ssd_debug_uniforms(int(seed) & ((1 << 64) - 1), B, W, _dev(out, "out"), _stream(stream)))
    return out


def read_status(workspace: Optional[torch.Tensor] = None, device=None, stream=None) -> int:
    """Read and clear the device status word (synchronises the stream)."""
    if workspace is None:
        workspace = _ws_cache.get(_ws_key(device))
        if workspace is None:
            return 0
    st = ctypes.c_int(0)
    _check(lib().ssd_read_status(_dev(workspace, "workspace"), workspace.numel(), ctypes.byref(st),
                                 _stream(stream)))
    return st.value
