"""Plain forms in 64 bits for the page plan, the norms and rotation, and attention whose rows see any set of
positions."""
import numpy as np
import torch


def plan(table, held, stack, n_free, length, new, page, shared):
    """The page plan, a page at a time; (table, held, stack, n_free, served) as arrays."""
    table, held, stack = table.copy(), held.copy(), stack.copy()
    free = stack[:n_free].tolist()
    B, width = table.shape
    ok = (length >= 0) & (new >= 0) & (length + new <= width * page) & (held >= 0) & (held <= width) & (shared >= 0) & \
        (shared <= held)
    hold = np.where(ok, np.maximum(shared, -(-(length + new) // page)), held)
    for b in range(B):
        for c in range(hold[b], held[b]):
            free.append(int(table[b, c]))
            table[b, c] = -1
    highest = len(free)
    served, short = ok.copy(), False
    for b in range(B):
        need = int(hold[b] - held[b])
        if need > 0:
            short = short or need > len(free)
            if short:
                served[b] = False
                continue
            for c in range(held[b], hold[b]):
                table[b, c] = free.pop()
        if served[b]:
            held[b] = hold[b]
    stack[:len(free)] = free
    stack[len(free):highest] = -1
    return table, held, stack, len(free), served


def slots(table, length, new, served, page, n):
    out = np.full((len(length), n), -1, dtype=np.int64)
    for b in range(len(length)):
        if served[b]:
            pos = int(length[b]) + np.arange(int(new[b]))
            out[b, :len(pos)] = table[b, pos // page] * page + pos % page
    return out


def rope(x, pos, weight, eps, freq, interleaved):
    """Rows x [n, heads, D] at positions pos [n]: (result, |a| + |b| of each element's pair)."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y * weight.astype(np.float64) / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    size = np.abs(y)
    if freq is not None:
        half = len(freq)
        t = pos[:, None].astype(np.float64) * freq.astype(np.float64)
        cos, sin = np.cos(t)[:, None], np.sin(t)[:, None]
        a = np.arange(half) * (2 if interleaved else 1)
        b = a + (1 if interleaved else half)
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * cos - v * sin, u * sin + v * cos
        size[..., a] = size[..., b] = np.abs(u) + np.abs(v)
    return y, size


def rope_bound(y, size, dtype):
    """|error| allowed: the sum of squares has 21 roundings, halved by the root, which with the division and the two
    products makes 15 halves of 2^-23; the angle is rounded once (pi 2^-24), sine and cosine are good to 2^-23, and
    the rotation rounds three times: 24 of 2^-24 in all, below 2^-19.  The output's own rounding is half a step."""
    return torch.finfo(dtype).eps / 2 * np.abs(y) * 1.01 + size * 2.0 ** -19 + 1e-37


def attend(q, k, v, seen, scale):
    """One request: q [n, H, D], k and v [T, Hkv, D] as held; seen(i): the positions that query i sees.
    (out, lse, mag, spread, count) as kv_common.attention gives them, and the sums of |v| over what is seen."""
    n, H, D = q.shape
    G = H // k.shape[1]
    out, mag = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, spread, count = np.full((n, H), -np.inf), np.zeros((n, H)), np.zeros((n, H))
    every = np.zeros((n, H, D))
    for i in range(n):
        at = seen(i)
        if len(at) == 0:
            continue
        for h in range(H):
            kk, vv = k[at, h // G], v[at, h // G]
            s = scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            out[i, h], lse[i, h] = (p @ vv) / z, m + np.log(z)
            mag[i, h] = (p @ np.abs(vv)) / z
            spread[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            count[i, h] = len(at)
            every[i, h] = np.abs(vv).sum(0)
    return (out, lse, mag, spread, count), every


def small_weights(every, dtype):
    """What rounding weights to fp16 adds to kv_common.bounds where the kernels keep no more than one pass of them.  A
    weight is 2^(x - m + 15) with m at least the row's largest score so far (fp32: two parts), or 2^(x - m + 9) with m at
    or below it (bf16 on the tensor cores).  Below 2^-14 fp16 numbers are multiples of 2^-24, so a
    weight is off by 2^-25 at most, which is 2^-40 or 2^-34 of the row's largest weight and no more of the sum of
    weights; each token's error comes with its |v|."""
    return every * (2.0 ** -40 if dtype == torch.float32 else 2.0 ** -34)
