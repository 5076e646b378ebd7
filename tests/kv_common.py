"""The 4-bit cache and its attention in 64 bits (numpy), from the definitions in
include/ssdv.h, with the error bounds the GPU tests hold the kernels to."""
import numpy as np
import torch

SCALES = np.array([m * 2.0 ** -17 for m in range(8)] +
                  [(8 + m) * 2.0 ** (e - 18) for e in range(1, 23) for m in range(8)])  # 0 .. 240
BORDERS = (SCALES[1:] + SCALES[:-1]) / 2


def held(x):
    """The values the cache holds for rows [..., D]."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    nan = np.isnan(g).any(-1, keepdims=True)
    a = np.where(nan, 0.0, np.abs(g)).max(-1, keepdims=True)
    at = np.searchsorted(7 * BORDERS, a)  # borders strictly below a
    tie = (at < len(BORDERS)) & (7 * BORDERS[np.minimum(at, len(BORDERS) - 1)] == a)
    s = SCALES[at + (tie & (at % 2 == 1))]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.where(s > 0, np.clip(np.rint(g / s), -7, 7), 0.0)
    return np.where(nan, np.nan, n * s).reshape(x.shape)


def attention(q, k, v, kv_len, n_q, scale, window=0, past_only=False):
    """One request: q [n, H, D], k and v [T, Hkv, D] as held.  (out, lse, bound, lse_bound): what any fp32 evaluation
    with 16-bit weights may differ by before its rounding to the output's type is in `bound_terms`."""
    n, H, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    out = np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    mag = np.zeros((n, H, D))  # sum p |v|
    spread = np.zeros((n, H))  # |scale| max_p sum_d |q k|
    count = np.zeros((n, H))
    for i in range(min(n, n_q)):
        pos = kv_len + i
        hi = kv_len if past_only else pos + 1
        lo = max(0, pos + 1 - window) if window else 0
        if lo >= hi:
            continue
        for h in range(H):
            kk, vv = k[lo:hi, h // G], v[lo:hi, h // G]
            s = scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            out[i, h] = (p @ vv) / z
            lse[i, h] = m + np.log(z)
            mag[i, h] = (p @ np.abs(vv)) / z
            spread[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            count[i, h] = hi - lo
    return out, lse, mag, spread, count


def bounds(out, lse, mag, spread, count, D, dtype):
    """|error| allowed.  Scores: D products summed in fp32 whose steps may truncate (2^-23 each, D / 16 fragments of 16
    summed at once, and 8 more for scaling and the exponential's argument); fp32 queries enter as two fp16 parts
    (2^-21).  Weights: fp16 (2^-11), for fp32 outputs two fp16 parts (2^-21); exponential 2^-21; what falls under the
    fp16 range of a weight is below 2^-30 of the largest.  Sums over tokens: one truncation per 16 tokens and 64 for
    joining parts.  The output's own rounding is half a step."""
    f32 = dtype == torch.float32
    e_score = spread * ((D / 16 + 8) * 2.0 ** -23 + (2.0 ** -21 if f32 else 0.0)) + np.abs(lse, where=np.isfinite(lse), out=np.zeros_like(lse)) * 2.0 ** -22
    e_sum = (count / 16 + 64) * 2.0 ** -23
    e_weight = (2.0 ** -21 if f32 else 2.0 ** -11) + 2.0 ** -21 + count * 2.0 ** -30
    rel = 2 * (np.exp(e_score) - 1) + 2 * e_sum + e_weight
    half = torch.finfo(dtype).eps / 2
    return half * np.abs(out) * 1.01 + rel[..., None] * mag + 1e-30, e_score + e_sum + 2.0 ** -21 + 2.0 ** -23 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


class Pool:
    """A cache on the GPU with shuffled pages for B requests, and the rows it should hold."""

    def __init__(self, ssdv, B, kv_heads, D, page, max_tokens, seed=0, fill=None, extra=3):
        g = np.random.default_rng(seed)
        self.ssdv, self.B, self.H, self.D, self.page = ssdv, B, kv_heads, D, page
        self.width = max(1, -(-max_tokens // page))
        n = B * self.width + extra
        self.cache = ssdv.make_kv_cache(n, kv_heads, D, page, device="cuda")
        if fill is not None:
            self.cache.fill_(fill)
        self.table = torch.from_numpy(g.permutation(n)[:B * self.width].reshape(B, self.width).astype(np.int32)).cuda()

    def append(self, start, k, v, n_new=None, **kw):
        self.ssdv.kv_append(self.cache, self.table, ints(start), k, v, n_new=None if n_new is None else ints(n_new), **kw)

    def read(self, start, n, dtype=torch.float32, count=None):
        k, v = self.ssdv.kv_read(self.cache, self.table, ints(start), n, dtype, count=None if count is None else ints(count))
        return k.double().cpu().numpy(), v.double().cpu().numpy()


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def rows(shape, dtype, seed, size=1.0):
    """Random rows whose channels differ in size, on the GPU, and their exact values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g)) * size
    x = x.to(dtype)
    return x.cuda(), x.double().numpy()
