"""Cases, plain forms and exact values for the 4-bit key/value cache: storing keys and values in it and reading them
back ("store"), and the attention of a verification round's query tokens over it ("attention").

The cache's numbers: 16 consecutive elements of a head's row form a group.  Its scale s is max|x| / 7 rounded to a
4-bit significand (to the nearest, ties to even; multiples of 2^-17 below 2^-14; at most 240), each element the
integer x / s rounded to the nearest (ties to even) and held to -7 .. 7.  A scale is one byte, the upper byte of an
fp16 number shifted to drop the sign: 5 bits of exponent, 3 of significand."""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 16


def listed():
    return [
        # one user, gamma = 5 drafts, a short chat: latency decides
        dict(name="verify_1_short", op="attention", batch=1, heads=32, kv_heads=8, dim=128, n_q=6, ragged_q=False,
             len_lo=707, len_hi=707, page=64, dtype="bf16", window=0, past_only=False),
        # the framework's main batch (64 requests, gamma = 4), 4 query heads a kv head, lengths far apart
        dict(name="verify_64_ragged", op="attention", batch=64, heads=32, kv_heads=8, dim=128, n_q=5, ragged_q=False,
             len_lo=201, len_hi=8003, page=64, dtype="bf16", window=0, past_only=False),
        # the same batch with 8 query heads a kv head: 40 rows share each key
        dict(name="verify_64_wide", op="attention", batch=64, heads=64, kv_heads=8, dim=128, n_q=5, ragged_q=False,
             len_lo=97, len_hi=4099, page=32, dtype="bf16", window=0, past_only=False),
        # two long documents: few rows, a long axis
        dict(name="verify_2_long", op="attention", batch=2, heads=64, kv_heads=8, dim=128, n_q=5, ragged_q=False,
             len_lo=99991, len_hi=131072, page=128, dtype="bf16", window=0, past_only=False),
        # no drafts: single-token decoding of a large batch
        dict(name="decode_128", op="attention", batch=128, heads=32, kv_heads=8, dim=128, n_q=1, ragged_q=False,
             len_lo=301, len_hi=6007, page=64, dtype="bf16", window=0, past_only=False),
        # the framework's ragged batch (512 requests, gamma 1..8), one shard of the heads, over the past alone, with
        # the log-sum-exps that join it to attention over the drafts' own unrounded keys; request 0 has no past
        dict(name="ragged_512_past", op="attention", batch=512, heads=8, kv_heads=2, dim=128, n_q=9, ragged_q=True,
             len_lo=0, len_hi=2503, page=16, dtype="bf16", window=0, past_only=True),
        # fp32, a head of keys per query head, a sliding window
        dict(name="window_f32", op="attention", batch=16, heads=16, kv_heads=16, dim=64, n_q=4, ragged_q=False,
             len_lo=1, len_hi=5003, page=64, dtype="f32", window=1024, past_only=False),
        # wide heads
        dict(name="verify_32_dim256", op="attention", batch=32, heads=16, kv_heads=8, dim=256, n_q=5, ragged_q=False,
             len_lo=513, len_hi=3001, page=64, dtype="bf16", window=0, past_only=False),
        # one round's gamma + 1 tokens of 64 requests, written inside partly filled blocks
        dict(name="append_round", op="store", batch=64, kv_heads=8, dim=128, page=64, dtype="bf16", len_lo=201,
             len_hi=8003, new_lo=5, new_hi=5, fused=True),
        # prompts of a few thousand tokens, k and v as slices of one projection's output
        dict(name="append_prompts", op="store", batch=8, kv_heads=8, dim=128, page=64, dtype="bf16", len_lo=0,
             len_hi=77, new_lo=701, new_hi=4099, fused=True),
        # one token of three requests in fp32: the smallest call
        dict(name="append_3_f32", op="store", batch=3, kv_heads=16, dim=64, page=16, dtype="f32", len_lo=15,
             len_hi=1001, new_lo=1, new_hi=1, fused=False),
        # ragged chunks into small pages, wide heads
        dict(name="append_300_dim256", op="store", batch=300, kv_heads=2, dim=256, page=32, dtype="bf16", len_lo=0,
             len_hi=509, new_lo=0, new_hi=41, fused=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """A case of the listed ranges; its cost is held below the largest listed case's."""
    dim = rng.choice([64, 128, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.35:
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        batch = _log_int(rng, 1, 300)
        new_hi = _log_int(rng, 1, 4100)
        while batch * new_hi * kv_heads * dim > 8 * 4096 * 8 * 128:
            batch, new_hi = max(1, batch // 2), max(1, new_hi // 2)
        return dict(op="store", batch=batch, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, len_lo=rng.randint(0, 40),
                    len_hi=rng.randint(40, 1200), new_lo=rng.randint(0, new_hi), new_hi=new_hi, fused=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    per = rng.choice([1, 2, 4, 5, 8])
    n_q = rng.randint(1, 9)
    batch = _log_int(rng, 1, 512)
    len_hi = _log_int(rng, 40, 131072)
    while (batch * len_hi * kv_heads * dim > 200000 * 8 * 128
           or 4.0 * batch * len_hi * kv_heads * dim * per * n_q > 3.5e10):
        if batch > 1:
            batch = batch // 2
        else:
            len_hi = len_hi // 2
    past_only = rng.random() < 0.3
    return dict(op="attention", batch=batch, heads=per * kv_heads, kv_heads=kv_heads, dim=dim, n_q=n_q,
                ragged_q=rng.random() < 0.4, len_lo=rng.randint(0, len_hi), len_hi=len_hi, page=page, dtype=dtype,
                window=rng.choice([0, 0, 0, rng.randint(1, 4096)]), past_only=past_only)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, spaced evenly in the logarithm: a case's lengths, whatever the seed."""
    if n == 1:
        return np.array([hi])
    t = np.linspace(0.0, 1.0, n)
    return np.rint((lo + 1) * ((hi + 1) / (lo + 1)) ** t).astype(np.int64) - 1


def _counts(case):
    """Per request: tokens before the call, tokens of the call."""
    n = case["batch"]
    before = _spread(case["len_lo"], case["len_hi"], n)
    if case["op"] == "store":
        lo, hi = case["new_lo"], case["new_hi"]
        new = lo + (np.arange(n) * 7 + 3) % (hi - lo + 1) if n > 1 else np.array([hi])
    elif case["ragged_q"]:
        new = 1 + (np.arange(n) * 5 + case["n_q"] - 1) % case["n_q"]
    else:
        new = np.full(n, case["n_q"])
    return before, new


def _visible(case, before, new):
    """Sum over requests of (keys that some query sees, query-key pairs)."""
    keys, pairs = 0, 0
    for length, m in zip(before.tolist(), new.tolist()):
        i = np.arange(m)
        hi = np.full(m, length) if case["past_only"] else length + i + 1
        lo = np.maximum(0, length + i + 1 - case["window"]) if case["window"] else np.zeros(m, dtype=np.int64)
        seen = np.maximum(hi - lo, 0)
        pairs += int(seen.sum())
        some = seen > 0
        if some.any():
            keys += int(hi[some].max() - lo[some].min())
    return keys, pairs


def work(case):
    before, new = _counts(case)
    size = 2 if case["dtype"] == "bf16" else 4
    dim, kv = case["dim"], case["kv_heads"]
    held = dim // 2 + dim // GROUP  # bytes of one row of one head in the cache
    if case["op"] == "store":
        rows = int(new.sum()) * kv * 2
        # read the rows, write them to the cache; read them there, write them out
        return {"bytes": rows * 2 * (dim * size + held), "flops": rows * dim * 6}
    keys, pairs = _visible(case, before, new)
    rows = int(new.sum()) * case["heads"]
    return {"bytes": keys * kv * 2 * held + rows * (2 * dim * size + 4), "flops": 4 * dim * case["heads"] * pairs}


def _inputs(case, seed):
    """What the model's projections give: keys with channels of unequal size and offset, values, queries whose logits
    spread by about two; the lengths in an order of the seed's."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    before, new = _counts(case)
    order = np.random.default_rng(seed).permutation(case["batch"])
    before, new = before[order], new[order]
    n, kv, dim = case["batch"], case["kv_heads"], case["dim"]
    if case["op"] == "store":
        start, count, longest = before, new, max(1, case["new_hi"])
    else:
        start = np.zeros_like(before)
        count = before if case["past_only"] else before + new
        longest = max(1, int(count.max()))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    size = torch.exp(0.5 * normal(kv, dim))
    shift = normal(kv, dim)

    def keys(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt).mul_(size.to(dt)).add_(shift.to(dt))

    if case.get("fused"):
        both = torch.empty(n, longest, 2, kv, dim, device="cuda", dtype=dt)
        both[:, :, 0] = keys(n, longest, kv, dim)
        both[:, :, 1] = torch.randn(n, longest, kv, dim, generator=gen, device="cuda", dtype=dt)
        k, v = both[:, :, 0], both[:, :, 1]
    else:
        k = keys(n, longest, kv, dim)
        v = torch.randn(n, longest, kv, dim, generator=gen, device="cuda", dtype=dt)
    out = dict(k=k, v=v, start=start, count=count, before=before, new=new)
    if case["op"] == "attention":
        out["q"] = (1.2 * normal(n, case["n_q"], case["heads"], dim)).to(dt)
    # pages in no order, some of the pool unused
    need = -(-(before + new) // case["page"])
    width = max(1, int(need.max()))
    pool = int(need.sum()) + 3
    ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = np.zeros((n, width), dtype=np.int64)
    at = 0
    for b in range(n):
        table[b, :need[b]] = np.arange(at, at + need[b])
        at += need[b]
    out["table"] = ids[torch.from_numpy(table).cuda()].contiguous()
    out["pool"] = pool
    return out


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


# ---- the plain form ---------------------------------------------------------------------------------------------

def _encode(x):
    """Rows [..., D] of any type to (packed codes [..., D/2], scale bytes [..., D/16])."""
    x = x.to(torch.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    top = g.abs().amax(-1)
    top = top / torch.full_like(top, 7.0)  # a true quotient: ties are ties
    _, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
    e = torch.where(top > 0, e - 4, torch.full_like(e, -17)).clamp_min(-17)
    step = torch.ldexp(torch.ones_like(top), e)
    s = (torch.round(top / step) * step).clamp_max(240.0)
    live = s > 0
    code = torch.round(g / torch.where(live, s, torch.ones_like(s)).unsqueeze(-1)).clamp(-7, 7)
    code = torch.where(live.unsqueeze(-1), code, torch.zeros_like(code)).to(torch.int32) + 8
    code = code.reshape(*x.shape[:-1], -1, 2)
    packed = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    m, e = torch.frexp(s)
    small = s < 2.0 ** -14
    byte = torch.where(small, torch.ldexp(s, torch.full_like(e, 17)),
                       8.0 * (e + 14).to(torch.float32) + torch.ldexp(m, torch.full_like(e, 4)) - 8.0)
    return packed, byte.to(torch.uint8)


def _decode(packed, byte):
    """The values held, in 32 bits."""
    p = packed.to(torch.int32)
    code = torch.stack([p % 16, p // 16], -1).reshape(*p.shape[:-1], -1, GROUP) - 8
    b = byte.to(torch.int32)
    e, m = b // 8, b % 8
    s = torch.where(e == 0, torch.ldexp(m.to(torch.float32), torch.full_like(e, -17)),
                    torch.ldexp((m + 8).to(torch.float32), e - 18))
    return (code.to(torch.float32) * s.unsqueeze(-1)).reshape(*p.shape[:-1], -1)


def _slots(case, table, start, count, longest):
    """For each request and each of its tokens: is it there, its page, its place in the page."""
    i = torch.arange(longest, device="cuda")
    pos = start.to(torch.int64)[:, None] + i
    there = i < count.to(torch.int64)[:, None]
    page = pos // case["page"]
    page = torch.where(there, page, torch.zeros_like(page)).clamp_max(table.shape[1] - 1)
    return there, torch.gather(table.to(torch.int64), 1, page), pos % case["page"]


def _plain_write(case, cache, table, start, count, k, v):
    step = max(1, (1 << 19) // (k.shape[1] * case["kv_heads"]))
    for b in range(0, k.shape[0], step):
        there, page, slot = _slots(case, table[b:b + step], start[b:b + step], count[b:b + step], k.shape[1])
        page, slot = page[there], slot[there]
        for name, x in (("k", k), ("v", v)):
            packed, byte = _encode(x[b:b + step][there])
            cache[name][page, slot] = packed
            cache[name + "s"][page, slot] = byte


def _plain_gather(case, cache, table, start, count, longest, name):
    there, page, slot = _slots(case, table, start, count, longest)
    x = _decode(cache[name][page, slot], cache[name + "s"][page, slot])
    return torch.where(there[..., None, None], x, torch.zeros_like(x))


def _plain_cache(case, pool):
    rows = (pool, case["page"], case["kv_heads"])
    cache = {}
    for name in ("k", "v"):
        cache[name] = torch.zeros(*rows, case["dim"] // 2, dtype=torch.uint8, device="cuda")
        cache[name + "s"] = torch.zeros(*rows, case["dim"] // GROUP, dtype=torch.uint8, device="cuda")
    return cache


def _plain_store(case, s):
    _plain_write(case, s["cache"], s["table"], s["start"], s["count"], s["k"], s["v"])
    dt = DTYPES[case["dtype"]]
    return [_plain_gather(case, s["cache"], s["table"], s["start"], s["count"], s["k"].shape[1], name).to(dt)
            for name in ("k", "v")]


def _plain_attention(case, s):
    q = s["q"]
    n, n_q, heads, dim = q.shape
    kv = case["kv_heads"]
    per = heads // kv
    longest = max(1, s["longest"])
    step = max(1, (1 << 20) // (longest * kv))
    out = torch.empty(n, n_q, heads, dim, device="cuda", dtype=q.dtype)
    lse = torch.empty(n, n_q, heads, device="cuda", dtype=torch.float32)
    for b in range(0, n, step):
        table, before, new = s["table"][b:b + step], s["before"][b:b + step], s["new"][b:b + step]
        count = before if case["past_only"] else before + new
        zero = torch.zeros_like(before)
        m = table.shape[0]
        k = _plain_gather(case, s["cache"], table, zero, count, longest, "k").permute(0, 2, 1, 3)
        x = q[b:b + step].to(torch.float32).reshape(m, n_q, kv, per, dim).permute(0, 2, 1, 3, 4)
        score = torch.matmul(x.reshape(m, kv, n_q * per, dim), k.transpose(2, 3)) / float(dim) ** 0.5
        del k
        at = before[:, None] + torch.arange(n_q, device="cuda")
        p = torch.arange(longest, device="cuda")
        seen = p < count[:, None, None]
        seen = seen & (p <= at[:, :, None]) & (torch.arange(n_q, device="cuda")[:, None] < new[:, None, None])
        if case["window"]:
            seen = seen & (p > at[:, :, None] - case["window"])
        seen = seen[:, None, :, None, :].expand(m, kv, n_q, per, longest).reshape(m, kv, n_q * per, longest)
        score = score.masked_fill(~seen, float("-inf"))
        top = score.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        weight = torch.exp(score - top)
        del score
        total = weight.sum(-1, keepdim=True)
        v = _plain_gather(case, s["cache"], table, zero, count, longest, "v").permute(0, 2, 1, 3)
        y = torch.matmul(weight, v) / torch.where(total > 0, total, torch.ones_like(total))
        z = (torch.log(total) + top).squeeze(-1)
        out[b:b + step] = y.reshape(m, kv, n_q, per, dim).permute(0, 2, 1, 3, 4).reshape(m, n_q, heads, dim).to(q.dtype)
        lse[b:b + step] = z.reshape(m, kv, n_q, per).permute(0, 2, 1, 3).reshape(m, n_q, heads)
    return [out, lse]


# ---- preparation and one pass -----------------------------------------------------------------------------------

def prepare(case, seed):
    """The cache (for attention already holding the keys and values), its page table, the lengths, and the call's
    own tensors.  A program that uses the plain form keeps the plain form of the cache."""
    x = _inputs(case, seed)
    s = dict(case=dict(case), table=x["table"], start=_ints(x["start"]), count=_ints(x["count"]),
             before=_ints(x["before"]), new=_ints(x["new"]), longest=int(x["count"].max()))
    if own:
        from speculative_decoding_verification_draft_gb300 import ssdv
        s["ssdv"] = ssdv
        s["cache"] = ssdv.make_kv_cache(x["pool"], case["kv_heads"], case["dim"], case["page"], device="cuda")
        if case["op"] == "attention":
            ssdv.kv_append(s["cache"], x["table"], s["start"], x["k"], x["v"], n_new=s["count"])
    else:
        s["cache"] = _plain_cache(case, x["pool"])
        if case["op"] == "attention":
            _plain_write(case, s["cache"], x["table"], s["start"], s["count"], x["k"], x["v"])
    if case["op"] == "attention":
        s["q"] = x["q"]
    else:
        s["k"], s["v"] = x["k"], x["v"]
    return s


def run(state):
    case = state["case"]
    if not own:
        return _plain_store(case, state) if case["op"] == "store" else _plain_attention(case, state)
    ssdv = state["ssdv"]
    if case["op"] == "store":
        ssdv.kv_append(state["cache"], state["table"], state["start"], state["k"], state["v"], n_new=state["count"])
        k, v = ssdv.kv_read(state["cache"], state["table"], state["start"], state["k"].shape[1],
                            DTYPES[case["dtype"]], count=state["count"])
        return [k, v]
    out, lse = ssdv.kv_attention(state["cache"], state["table"], state["before"], state["q"], n_q=state["new"],
                                 window=case["window"], past_only=case["past_only"], return_lse=True)
    return [out, lse]


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def _scale_table():
    """Every scale from 0 to 240, and the borders between neighbours."""
    values = [m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 23) for m in range(8)]
    values = torch.tensor(values, dtype=torch.float64, device="cuda")
    return values, (values[1:] + values[:-1]) / 2


def _held(x):
    """The value that the cache holds for each element of rows [..., D], in 64 bits."""
    values, borders = _scale_table()
    g = x.to(torch.float64).reshape(*x.shape[:-1], -1, GROUP)
    top = g.abs().amax(-1)
    # compare 7 border with the maximum: both are exact in 64 bits
    at = torch.searchsorted(borders * 7.0, top)  # number of borders below top
    tie = (at < borders.numel()) & (borders[at.clamp_max(borders.numel() - 1)] * 7.0 == top)
    at = at + (tie & (at % 2 == 1)).to(at.dtype)
    s = values[at].unsqueeze(-1)
    code = torch.where(s > 0, g / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    return (code.round().clamp(-7, 7) * s).reshape(x.shape)


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "store":
        there = torch.arange(x["k"].shape[1], device="cuda") < _ints(x["count"])[:, None]
        return [torch.where(there[..., None, None], _held(x[name]), torch.zeros((), dtype=torch.float64, device="cuda"))
                for name in ("k", "v")]
    q = x["q"].to(torch.float64)
    n, n_q, heads, dim = q.shape
    per = heads // case["kv_heads"]
    out = torch.zeros(n, n_q, heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((n, n_q, heads), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(n):
        count, before, new = int(x["count"][b]), int(x["before"][b]), int(x["new"][b])
        if count == 0 or new == 0:
            continue
        row = before + torch.arange(new, device="cuda")[:, None]
        p = torch.arange(count, device="cuda")
        hidden = p > row
        if case["window"]:
            hidden = hidden | (p <= row - case["window"])
        k, v = _held(x["k"][b, :count]), _held(x["v"][b, :count])
        for h in range(case["kv_heads"]):
            mine = slice(h * per, (h + 1) * per)
            score = torch.einsum("iad,pd->aip", q[b, :new, mine], k[:, h]) * dim ** -0.5
            score[:, hidden] = float("-inf")
            z = torch.logsumexp(score, -1)
            weight = torch.where(torch.isinf(z)[..., None], torch.zeros_like(score), torch.exp(score - z[..., None]))
            out[b, :new, mine] = torch.einsum("aip,pd->iad", weight, v[:, h])
            lse[b, :new, mine] = z.transpose(0, 1)
    return [out, lse]
