"""Cases, plain forms and exact values for what a round needs around the 4-bit key/value cache:

  plan    the page table and the slots of the new tokens, from the requests' lengths and a stack of free pages
  rope    norms of queries and keys for each head, with the rotation by position
  sinks   attention over the cache within a window, with a few first tokens that stay visible
  shared  attention over the cache for requests that share a long prefix

The cache's numbers: 16 consecutive elements of a head's row form a group.  Its scale s is max|x| / 7 rounded to a
4-bit significand (to the nearest, ties to even; multiples of 2^-17 below 2^-14; at most 240), each element the
integer x / s rounded to the nearest (ties to even) and held to -7 .. 7."""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 16
EPS = 1e-6
THETA = 500000.0


def listed():
    return [
        # a round of the framework's main batch: five more tokens each, now and then a page; two requests have ended,
        # two begin
        dict(name="plan_64_round", op="plan", batch=64, page=64, len_lo=201, len_hi=8003, n=5, done=2, prompts=2,
             prompt_hi=1500, shared=0, tight=False),
        # a large batch with many prompts to place behind a shared prefix, and not enough free pages for all of them
        dict(name="plan_512_prompts", op="plan", batch=512, page=16, len_lo=33, len_hi=4099, n=5, done=61, prompts=97,
             prompt_hi=2047, shared=6, tight=True),
        # one new token of three requests in fp32, a head of keys per query head: the smallest call
        dict(name="rope_3_f32", op="rope", batch=3, n=1, ragged=False, heads=16, kv_heads=16, dim=64, rot=64,
             interleaved=False, norm=True, dtype="f32", len_lo=15, len_hi=130003, fused=False),
        # gamma + 1 tokens of the main batch, queries and keys slices of one projection
        dict(name="rope_64_round", op="rope", batch=64, n=5, ragged=False, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, dtype="bf16", len_lo=201, len_hi=8003, fused=True),
        # prompts of a few thousand tokens, a quarter of each wide head rotated, pairs side by side
        dict(name="rope_prompts", op="rope", batch=8, n=4099, ragged=True, heads=16, kv_heads=8, dim=256, rot=64,
             interleaved=True, norm=True, dtype="bf16", len_lo=0, len_hi=77, fused=True),
        # fp32, a short window, requests of no token among them, ragged query counts
        dict(name="sinks_16_f32", op="sinks", batch=16, heads=16, kv_heads=16, dim=64, n=4, ragged=True, len_lo=0,
             len_hi=3001, window=255, sinks=3, page=64, dtype="f32", past_only=False),
        # the main batch: 64 requests, gamma = 4, four first tokens
        dict(name="sinks_64_round", op="sinks", batch=64, heads=32, kv_heads=8, dim=128, n=5, ragged=False, len_lo=201,
             len_hi=8003, window=1024, sinks=4, page=64, dtype="bf16", past_only=False),
        # no drafts: single tokens of a large batch, a wide window and a block of first tokens
        dict(name="sinks_128_decode", op="sinks", batch=128, heads=32, kv_heads=8, dim=128, n=1, ragged=False,
             len_lo=301, len_hi=9001, window=4096, sinks=64, page=64, dtype="bf16", past_only=False),
        # fp32, two short shared prefixes of odd lengths
        dict(name="shared_6_f32", op="shared", batch=6, groups=2, heads=8, kv_heads=4, dim=64, n=3, ragged=True,
             pre_lo=331, pre_hi=777, own_lo=0, own_hi=90, page=16, dtype="f32", past_only=False),
        # 16 prompts, 8 samples of each, one token at a time: 32 rows a group and kv head
        dict(name="shared_16x8_samples", op="shared", batch=128, groups=16, heads=32, kv_heads=8, dim=128, n=1,
             ragged=False, pre_lo=301, pre_hi=6007, own_lo=1, own_hi=701, page=64, dtype="bf16", past_only=False),
        # the main batch behind one system prompt: 1280 rows a kv head
        dict(name="shared_64_system", op="shared", batch=64, groups=1, heads=32, kv_heads=8, dim=128, n=5, ragged=False,
             pre_lo=4096, pre_hi=4096, own_lo=33, own_hi=1025, page=64, dtype="bf16", past_only=False),
        # 256 requests on one long document, 8 query heads a kv head
        dict(name="shared_256_document", op="shared", batch=256, groups=1, heads=64, kv_heads=8, dim=128, n=5,
             ragged=True, pre_lo=16001, pre_hi=16001, own_lo=5, own_hi=803, page=64, dtype="bf16", past_only=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """A case of the listed ranges; its cost is held below the largest listed case's of its kind."""
    op = rng.choice(["plan", "rope", "sinks", "shared"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        batch = _log_int(rng, 1, 512)
        done = rng.randint(0, batch // 4)
        return dict(op=op, batch=batch, page=page, len_lo=rng.randint(0, 100), len_hi=_log_int(rng, 101, 4099),
                    n=rng.randint(1, 9), done=done, prompts=rng.randint(0, batch // 4), prompt_hi=_log_int(rng, 10, 2047),
                    shared=rng.choice([0, 0, 3, 6]), tight=rng.random() < 0.3)
    if op == "rope":
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        per = rng.choice([1, 2, 3, 4, 8])
        batch, n = _log_int(rng, 1, 300), _log_int(rng, 1, 4099)
        while batch * n * kv_heads * (per + 1) * dim > 8 * 4099 * 24 * 256 // 2:
            batch, n = max(1, batch // 2), max(1, n // 2)
        norm = rng.random() < 0.8
        return dict(op=op, batch=batch, n=n, ragged=rng.random() < 0.4, heads=per * kv_heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([16, 32, 64, dim, dim] + [0] * norm), interleaved=rng.random() < 0.4, norm=norm,
                    dtype=dtype, len_lo=rng.randint(0, 100), len_hi=_log_int(rng, 101, 1000003),
                    fused=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    per = rng.choice([1, 2, 4, 5, 8])
    n = rng.randint(1, 9)
    both = dict(op=op, heads=per * kv_heads, kv_heads=kv_heads, dim=dim, n=n, ragged=rng.random() < 0.4, page=page,
                dtype=dtype, past_only=rng.random() < 0.3)
    if op == "sinks":
        batch, len_hi = _log_int(rng, 1, 300), _log_int(rng, 40, 40009)
        while batch * len_hi * kv_heads * dim > 300000 * 8 * 128:
            batch, len_hi = (batch // 2, len_hi) if batch > 1 else (batch, len_hi // 2)
        return dict(both, batch=batch, len_lo=rng.randint(0, len_hi), len_hi=len_hi, window=_log_int(rng, 1, 4096),
                    sinks=_log_int(rng, 1, 130))
    batch = _log_int(rng, 2, 256)
    groups = _log_int(rng, 1, batch)
    pre_hi, own_hi = _log_int(rng, 20, 16001), _log_int(rng, 4, 803)
    # (products in fp32 cost several times those of the wider type; a wide head costs the kernels of either more)
    while (batch * pre_hi * kv_heads * per * n * dim > 256 * 16001 * 64 * 5 * 128 // (8 if dtype == "f32" or dim == 256 else 1)
           or (groups * pre_hi + batch * own_hi) * kv_heads * dim > 200000 * 8 * 128):
        if batch > 2 and batch * n * per > 64:
            batch = batch // 2
        else:
            pre_hi, own_hi = max(2, pre_hi // 2), max(2, own_hi // 2)
        groups = min(groups, batch)
    return dict(both, batch=batch, groups=groups, pre_lo=rng.randint(1, pre_hi), pre_hi=pre_hi,
                own_lo=rng.randint(0, own_hi // 2), own_hi=own_hi)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, spaced evenly in the logarithm: a case's lengths, whatever the seed."""
    if n == 1:
        return np.array([hi])
    t = np.linspace(0.0, 1.0, n)
    return np.rint((lo + 1) * ((hi + 1) / (lo + 1)) ** t).astype(np.int64) - 1


def _new(case):
    """Tokens of the call, request by request."""
    n, b = case["n"], case["batch"]
    if case["ragged"]:
        return 1 + (np.arange(b) * 5 + n - 1) % n if case["op"] != "rope" else 1 + (np.arange(b) * 7919 + n - 1) % n
    return np.full(b, n)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _seen(case, before, new):
    """Sum over requests of (keys that some query sees, query-key pairs) with a window and sinks."""
    keys = pairs = 0
    for length, m in zip(before.tolist(), new.tolist()):
        i = np.arange(m)
        hi = np.full(m, length) if case["past_only"] else length + i + 1
        lo = np.clip(length + i + 1 - case["window"], 0, hi)
        first = np.minimum(case["sinks"], lo)  # sinks that lie before the window
        pairs += int((hi - lo + first).sum())
        keys += int(hi.max() - lo.min() + first.min())
    return keys, pairs


def work(case):
    if case["op"] == "plan":
        x = _plan_lengths(case)
        b, width = case["batch"], x["width"]
        # lengths, counts and held pages read; table, stack and counts written beside what they were; a slot a token
        return {"bytes": 4 * (4 * b + 2 * b * width + 2 * x["pool"] + b + 2) + 8 * b * x["n"], "flops": 8 * b * (width + x["n"])}
    size = 2 if case["dtype"] == "bf16" else 4
    new = _new(case)
    dim, heads, kv = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "rope":
        count = int(new.sum()) * (heads + kv) * dim
        written = case["batch"] * case["n"] * (heads + kv) * dim
        return {"bytes": (count + written) * size + 8 * case["batch"] + 8 * dim, "flops": count * 8}
    held = dim // 2 + dim // GROUP  # bytes of one row of one head in the cache
    rows = int(new.sum()) * heads
    if case["op"] == "sinks":
        keys, pairs = _seen(case, _spread(case["len_lo"], case["len_hi"], case["batch"]), new)
    else:
        x = _shared_lengths(case)
        keys = int(x["pre"].sum() + (x["own"] + (0 if case["past_only"] else x["new"])).sum())
        past = x["new"] * (x["pre"][x["group"]] + x["own"])
        pairs = int(past.sum() + (0 if case["past_only"] else (x["new"] * (x["new"] + 1) // 2).sum()))
    return {"bytes": keys * kv * 2 * held + rows * (2 * dim * size + 4), "flops": 4 * dim * heads * pairs}


# ---- the cache's numbers, plain -----------------------------------------------------------------------------------

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
    byte = torch.where(s < 2.0 ** -14, torch.ldexp(s, torch.full_like(e, 17)),
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


def _plain_cache(case, pool):
    """Codes and scales [pool * page, kv_heads, ...], a row a slot."""
    rows = (pool * case["page"], case["kv_heads"])
    return {name + part: torch.zeros(*rows, case["dim"] // size, dtype=torch.uint8, device="cuda")
            for name in ("k", "v") for part, size in (("", 2), ("s", GROUP))}


def _slots(case, table, pos):
    """Slots of the positions pos [B, n] (those past the table's width: of its last column)."""
    page = torch.gather(table.to(torch.int64), 1, (pos // case["page"]).clamp_max(table.shape[1] - 1))
    return page * case["page"] + pos % case["page"]


def _plain_write(case, cache, table, start, count, k, v):
    step = max(1, (1 << 19) // (k.shape[1] * case["kv_heads"]))
    i = torch.arange(k.shape[1], device="cuda")
    for b in range(0, k.shape[0], step):
        there = i < count[b:b + step].to(torch.int64)[:, None]
        slot = _slots(case, table[b:b + step], start[b:b + step].to(torch.int64)[:, None] + i)[there]
        for name, x in (("k", k), ("v", v)):
            packed, byte = _encode(x[b:b + step][there])
            cache[name][slot] = packed
            cache[name + "s"][slot] = byte


def _plain_gather(cache, slot, name):
    return _decode(cache[name][slot], cache[name + "s"][slot])


# ---- plan ---------------------------------------------------------------------------------------------------------

def _plan_lengths(case):
    """Each request's state in the order of a batch: going on, ended, or beginning with a prompt."""
    b, page, shared = case["batch"], case["page"], case["shared"]
    length = shared * page + _spread(case["len_lo"], case["len_hi"], b)
    new = 1 + (np.arange(b) * 3) % case["n"]
    held = np.maximum(shared, -(-length // page))  # what the last round left: up to its last token
    at = (np.arange(b) * 89 + 5) % b if b % 89 else np.arange(b)
    end, begin = at[:case["done"]], at[case["done"]:case["done"] + case["prompts"]]
    length[end] = new[end] = 0
    held[begin], length[begin] = shared, shared * page
    new[begin] = 1 + (np.arange(len(begin)) * 613 + case["prompt_hi"] - 1) % case["prompt_hi"]
    hold = np.maximum(shared, -(-(length + new) // page))
    want, give = int(np.maximum(hold - held, 0).sum()), int(np.maximum(held - hold, 0).sum())
    free = max(0, want * 2 // 3 - give) if case["tight"] else want + 37
    own_pages = int((held - shared).sum())
    return dict(length=length, new=new, held=held, free=free, pool=shared + own_pages + free, n=int(new.max()),
                width=int(max(held.max(), hold.max())) + 3)


def _plan_inputs(case, seed):
    x = _plan_lengths(case)
    rng = np.random.default_rng(seed)
    order = rng.permutation(case["batch"])
    length, new, held = (x[k][order] for k in ("length", "new", "held"))
    ids = rng.permutation(x["pool"])
    shared = case["shared"]
    table = np.full((case["batch"], x["width"]), -1)
    col = np.arange(x["width"])
    table[:, :shared] = ids[:shared]
    mine = (col >= shared) & (col < held[:, None])
    table[mine] = ids[shared:shared + int(mine.sum())]
    stack = np.full(x["pool"], -1)
    stack[:x["free"]] = ids[shared + int(mine.sum()):]
    return dict(length=length, new=new, held=held, table=table, stack=stack, free=np.array([x["free"]]), n=x["n"])


def _plain_plan(case, s):
    page, shared = case["page"], case["shared"]
    length, new, held, table = (s[k].to(torch.int64) for k in ("length", "new", "held", "table"))
    hold = ((length + new + page - 1) // page).clamp_min(shared)
    give, want = (held - hold).clamp_min(0), (hold - held).clamp_min(0)
    n_free, pool = s["free"].to(torch.int64), s["stack"].numel()
    total = n_free + give.sum()  # pages on the stack once all that is given back lies on it
    served = (want.cumsum(0) <= total) | (want == 0)
    want = torch.where(served, want, torch.zeros_like(want))
    taken = want.sum()
    after = torch.where(served, hold, held)
    col = torch.arange(table.shape[1], device="cuda")
    back = (col >= after[:, None]) & (col < held[:, None])
    take = (col >= held[:, None]) & (col < after[:, None])
    # given back in the order of requests and columns, on top of the stack (one place more takes what is not)
    rank = give.cumsum(0)[:, None] - give[:, None] + col - after[:, None]
    stack = torch.cat([s["stack"].to(torch.int64), torch.full((1,), -1, device="cuda")])
    at = torch.where(back, n_free + rank, torch.full_like(rank, pool))
    stack = stack.scatter(0, at.reshape(-1), table.reshape(-1))
    # taken from the top, in the same order
    rank = want.cumsum(0)[:, None] - want[:, None] + col - held[:, None]
    at = torch.where(take, total - 1 - rank, torch.full_like(rank, pool))
    table = torch.where(take, stack[at], torch.where(back, torch.full_like(table, -1), table))
    left = total - taken
    i = torch.arange(pool, device="cuda")
    stack = torch.where(i < left, stack[:pool], torch.full_like(i, -1))
    i = torch.arange(s["n"], device="cuda")
    pos = length[:, None] + i
    slot = _slots(case, table, pos)
    slot = torch.where((i < new[:, None]) & served[:, None], slot, torch.full_like(slot, -1))
    return [table.to(torch.int32), after.to(torch.int32), stack.to(torch.int32), left.to(torch.int32), slot]


def _exact_plan(case, seed):
    """The same, page by page."""
    x = _plan_inputs(case, seed)
    page, shared = case["page"], case["shared"]
    table, held = x["table"].copy(), x["held"].copy()
    stack = x["stack"][:int(x["free"][0])].tolist()
    hold = [max(shared, -(-int(a + b) // page)) for a, b in zip(x["length"], x["new"])]
    slot = np.full((case["batch"], x["n"]), -1, dtype=np.int64)
    for b, h in enumerate(hold):
        for c in range(h, int(held[b])):
            stack.append(int(table[b, c]))
            table[b, c] = -1
        held[b] = min(held[b], h)
    short = False
    for b, h in enumerate(hold):
        need = h - int(held[b])
        short = short or need > len(stack)
        if need and short:
            continue
        for c in range(int(held[b]), h):
            table[b, c] = stack.pop()
        held[b] = h
        pos = int(x["length"][b]) + np.arange(int(x["new"][b]))
        slot[b, :len(pos)] = table[b, pos // page] * page + pos % page
    out = np.full(len(x["stack"]), -1)
    out[:len(stack)] = stack
    return [torch.from_numpy(np.ascontiguousarray(a)) for a in (table, held, out, np.array([len(stack)]), slot)]


# ---- rope ---------------------------------------------------------------------------------------------------------

def _rope_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, n, heads, kv, dim = case["batch"], case["n"], case["heads"], case["kv_heads"], case["dim"]
    dt = DTYPES[case["dtype"]]
    order = rng.permutation(b)
    # heads and channels of unequal size, as projections give them
    size = torch.exp(0.5 * torch.randn(heads + 2 * kv, dim, generator=gen, device="cuda"))
    if case["fused"]:
        x = torch.randn(b, n, heads + 2 * kv, dim, generator=gen, device="cuda", dtype=dt).mul_(size.to(dt))
        q, k = x[:, :, :heads], x[:, :, heads:heads + kv]
    else:
        q = torch.randn(b, n, heads, dim, generator=gen, device="cuda", dtype=dt).mul_(size[:heads].to(dt))
        k = torch.randn(b, n, kv, dim, generator=gen, device="cuda", dtype=dt).mul_(size[heads:heads + kv].to(dt))
    half = case["rot"] // 2
    freq = torch.from_numpy(THETA ** (-np.arange(half) / max(half, 1))).to(torch.float32).cuda() if half else None
    weight = [1.0 + 0.3 * torch.randn(dim, generator=gen, device="cuda") for _ in range(2)] if case["norm"] else [None, None]
    return dict(q=q, k=k, length=_ints(_spread(case["len_lo"], case["len_hi"], b)[order]), new=_ints(_new(case)[order]),
                freq=freq, weight=weight)


def _plain_rope(case, s):
    n, half = case["n"], case["rot"] // 2
    i = torch.arange(n, device="cuda")
    there = (i < s["new"].to(torch.int64)[:, None])[..., None, None]
    if half:
        # angles of far positions in 64 bits
        angle = (s["length"].to(torch.float64)[:, None] + i)[..., None] * s["freq"].to(torch.float64)
        cos, sin = torch.cos(angle).to(torch.float32)[:, :, None], torch.sin(angle).to(torch.float32)[:, :, None]
    out = []
    for x, weight in ((s["q"], s["weight"][0]), (s["k"], s["weight"][1])):
        dt = x.dtype
        x = x.to(torch.float32)
        if weight is not None:
            x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * weight
        if half:
            turn, rest = x[..., :2 * half], x[..., 2 * half:]
            if case["interleaved"]:
                a, b = turn[..., 0::2], turn[..., 1::2]
                turn = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
            else:
                a, b = turn[..., :half], turn[..., half:]
                turn = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
            x = torch.cat([turn, rest], -1)
        out.append(torch.where(there, x, torch.zeros((), device="cuda")).to(dt))
    return out


def _exact_rope(case, seed):
    x = _rope_inputs(case, seed)
    half = case["rot"] // 2
    out = []
    for rows, weight in ((x["q"], x["weight"][0]), (x["k"], x["weight"][1])):
        y = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            m = int(x["new"][b])
            r = rows[b, :m].to(torch.float64)
            if weight is not None:
                r = r * weight.to(torch.float64) * (r.square().sum(-1, keepdim=True) / case["dim"] + EPS).rsqrt()
            if half:
                pos = int(x["length"][b]) + torch.arange(m, device="cuda", dtype=torch.float64)
                z = torch.polar(torch.ones(m, half, dtype=torch.float64, device="cuda"), torch.outer(pos, x["freq"].to(torch.float64)))
                first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
                second = first + (1 if case["interleaved"] else half)
                turned = torch.complex(r[..., first], r[..., second]) * z[:, None]
                r[..., first], r[..., second] = turned.real, turned.imag
            y[b, :m] = r
        out.append(y)
    return out


# ---- sinks and shared: inputs -------------------------------------------------------------------------------------

def _pages(counts, page, gen, extra=3):
    """Tables of pages in no order for rows that hold counts[b] pages each, and the pool's size."""
    width, pool = max(1, int(counts.max())), int(counts.sum()) + extra
    ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = np.zeros((len(counts), width), dtype=np.int64)
    at = np.cumsum(counts) - counts
    for b in range(len(counts)):
        table[b, :counts[b]] = at[b] + np.arange(counts[b])
    return ids[torch.from_numpy(table).cuda()].contiguous(), pool


class _Rows:
    """Keys, values and queries as a model's projections give them: channels of unequal size, logits that spread by
    about two.  Sinks are keys along a direction that the queries share, with small values."""

    def __init__(self, case, gen):
        self.gen, self.dt, self.kv, self.dim, self.heads = gen, DTYPES[case["dtype"]], case["kv_heads"], case["dim"], case["heads"]
        self.size = torch.exp(0.5 * self.normal(self.kv, self.dim)).to(self.dt)
        self.shift = self.normal(self.kv, self.dim).to(self.dt)
        way = self.normal(self.kv, self.dim)
        self.way = way / way.square().sum(-1, keepdim=True).sqrt() * float(self.dim) ** 0.25

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.gen, device="cuda", dtype=dtype)

    def keys(self, *shape):
        return self.normal(*shape, self.kv, self.dim, dtype=self.dt).mul_(self.size).add_(self.shift)

    def values(self, *shape):
        return self.normal(*shape, self.kv, self.dim, dtype=self.dt)

    def sink(self, k, v, n):
        """The first n tokens draw weight: scores some ten above the others'."""
        k[:, :n] += (5.0 * self.way).to(self.dt)
        v[:, :n] *= 0.1

    def queries(self, b, n):
        q = 1.2 * self.normal(b, n, self.heads, self.dim)
        return (q + 2.0 * self.way.repeat_interleave(self.heads // self.kv, 0)).to(self.dt)


def _sinks_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = np.random.default_rng(seed).permutation(case["batch"])
    before, new = _spread(case["len_lo"], case["len_hi"], case["batch"])[order], _new(case)[order]
    count = before if case["past_only"] else before + new
    longest = max(1, int(count.max()))
    rows = _Rows(case, gen)
    k, v = rows.keys(case["batch"], longest), rows.values(case["batch"], longest)
    rows.sink(k, v, min(case["sinks"], 4))
    table, pool = _pages(-(-(before + new) // case["page"]), case["page"], gen)
    return dict(k=k, v=v, q=rows.queries(case["batch"], case["n"]), before=before, new=new, count=count, table=table,
                pool=pool)


def _shared_lengths(case):
    b, g = case["batch"], case["groups"]
    cut = np.arange(g + 1) * b // g
    group = np.repeat(np.arange(g), np.diff(cut))
    own_len = _spread(case["own_lo"], case["own_hi"], b)[(np.arange(b) * 37 + 1) % b if b % 37 else np.arange(b)]
    return dict(start=cut, group=group, pre=_spread(case["pre_lo"], case["pre_hi"], g), own=own_len, new=_new(case))


def _shared_inputs(case, seed):
    """Every group's prefix, every request's own tokens.  Pages that the prefix fills are shared; a page that it fills
    in part is the request's own, with the prefix's last tokens in it."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = _shared_lengths(case)
    rng = np.random.default_rng(seed)
    x["pre"] = x["pre"][rng.permutation(case["groups"])]
    order = rng.permutation(case["batch"])
    x["own"], x["new"] = x["own"][order], x["new"][order]
    page, group = case["page"], x["group"]
    before = x["pre"][group] + x["own"]
    count = before if case["past_only"] else before + x["new"]
    rows = _Rows(case, gen)
    pk, pv = rows.keys(case["groups"], int(x["pre"].max())), rows.values(case["groups"], int(x["pre"].max()))
    rows.sink(pk, pv, 1)
    # pages: those that the prefixes fill, then each request's own
    full = x["pre"] // page
    n_pages = -(-(before + x["new"]) // page)
    mine = n_pages - full[group]
    width, pool = max(1, int(n_pages.max())), int(full.sum() + mine.sum()) + 3
    ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = np.zeros((case["batch"], width), dtype=np.int64)
    first = np.cumsum(full) - full
    at = int(full.sum())
    for b, g in enumerate(group):
        table[b, :full[g]] = first[g] + np.arange(full[g])
        table[b, full[g]:n_pages[b]] = at + np.arange(mine[b])
        at += mine[b]
    # what a request writes itself: from the first page that it does not share
    begin = full[group] * page
    tail, longest = x["pre"][group] - begin, max(1, int((count - begin).max()))
    k, v = rows.keys(case["batch"], longest), rows.values(case["batch"], longest)
    for b, g in enumerate(group):
        for mine_, theirs in ((k, pk), (v, pv)):
            mine_[b, :tail[b]] = theirs[g, begin[b]:x["pre"][g]]
    return dict(x, pk=pk, pv=pv, k=k, v=v, q=rows.queries(case["batch"], case["n"]), before=before, count=count,
                begin=begin, table=ids[torch.from_numpy(table).cuda()].contiguous(), pool=pool)


# ---- sinks and shared: plain --------------------------------------------------------------------------------------

def _softmax_sums(score, seen):
    """(weights, their reference, their sums) of scores [..., rows, tokens]; a row that sees nothing has sum 0."""
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weight = torch.exp(score - top)
    return weight, top, weight.sum(-1, keepdim=True)


def _plain_sinks(case, s):
    q, window, sinks = s["q"], case["window"], case["sinks"]
    b, n, heads, dim = q.shape
    kv = case["kv_heads"]
    per = heads // kv
    longest = max(1, s["longest"])
    step = max(1, (1 << 20) // (min(longest, window + n + sinks) * kv))
    out = torch.empty_like(q)
    lse = torch.empty(b, n, heads, device="cuda", dtype=torch.float32)
    for at in range(0, b, step):
        table, before, new = (s[x][at:at + step].to(torch.int64) for x in ("table", "before", "new"))
        m = table.shape[0]
        row = before[:, None] + torch.arange(n, device="cuda")  # positions of the queries
        # what some query of the request may see: the sinks, then the window of the first query on
        first = torch.arange(sinks, device="cuda").expand(m, sinks)
        begin = (before + 1 - window).clamp_min(sinks)
        rest = begin[:, None] + torch.arange(min(longest, window + n), device="cuda")
        pos = torch.cat([first, rest], 1)
        hi = before[:, None].expand(m, n) if case["past_only"] else row + 1
        seen = (pos[:, None] < hi[..., None]) & ((pos[:, None] < sinks) | (pos[:, None] > row[..., None] - window))
        seen = seen & (torch.arange(n, device="cuda") < new[:, None])[..., None]
        slot = _slots(case, table, pos)
        slot = torch.where(pos < (before if case["past_only"] else before + new)[:, None], slot, torch.zeros_like(slot))
        k = _plain_gather(s["cache"], slot, "k").permute(0, 2, 3, 1)
        x = q[at:at + step].to(torch.float32).reshape(m, n, kv, per, dim).permute(0, 2, 1, 3, 4).reshape(m, kv, n * per, dim)
        score = torch.matmul(x, k) / float(dim) ** 0.5
        seen = seen[:, None, :, None].expand(m, kv, n, per, pos.shape[1]).reshape(score.shape)
        weight, top, total = _softmax_sums(score, seen)
        v = _plain_gather(s["cache"], slot, "v").permute(0, 2, 1, 3)
        y = torch.matmul(weight, v) / torch.where(total > 0, total, torch.ones_like(total))
        z = (torch.log(total) + top).squeeze(-1)
        out[at:at + step] = y.reshape(m, kv, n, per, dim).permute(0, 2, 1, 3, 4).reshape(m, n, heads, dim).to(q.dtype)
        lse[at:at + step] = z.reshape(m, kv, n, per).permute(0, 2, 1, 3).reshape(m, n, heads)
    return [out, lse]


def _plain_shared(case, s):
    """Each group's prefix against all rows of the group, each request's own tokens against its rows."""
    q = s["q"]
    b, n, heads, dim = q.shape
    kv = case["kv_heads"]
    per = heads // kv
    out = torch.zeros_like(q)
    lse = torch.empty(b, n, heads, device="cuda", dtype=torch.float32)
    i = torch.arange(n, device="cuda")
    for g, (lo, hi) in enumerate(zip(s["cut"][:-1], s["cut"][1:])):
        m, pre = hi - lo, s["pre"][g]
        table, before, new = (s[x][lo:hi].to(torch.int64) for x in ("table", "before", "new"))
        x = q[lo:hi].to(torch.float32).reshape(m, n, kv, per, dim).permute(2, 0, 1, 3, 4).reshape(kv, m, n * per, dim)
        real = (i < new[:, None])[:, :, None].expand(m, n, per).reshape(1, m, n * per, 1)
        slot = _slots(case, table[:1], torch.arange(pre, device="cuda")[None])[0]
        k, v = (_plain_gather(s["cache"], slot, name).permute(1, 0, 2) for name in ("k", "v"))
        longest = s["own"][g] + (0 if case["past_only"] else n)
        pos = pre + torch.arange(longest, device="cuda")[None].expand(m, longest)
        own_slot = _slots(case, table, pos)
        there = pos < (before if case["past_only"] else before + new)[:, None]
        own_slot = torch.where(there, own_slot, torch.zeros_like(own_slot))
        row = before[:, None] + i
        seen = pos[:, None] < (before[:, None, None] if case["past_only"] else row[..., None] + 1)
        seen = seen[:, :, None].expand(m, n, per, longest).reshape(1, m, n * per, longest)
        ok, ov = (_plain_gather(s["cache"], own_slot, name).permute(2, 0, 1, 3) for name in ("k", "v"))
        for h in range(kv):
            far = torch.matmul(x[h].reshape(-1, dim), k[h].transpose(0, 1)) / float(dim) ** 0.5
            near = torch.matmul(x[h], ok[h].transpose(1, 2)) / float(dim) ** 0.5
            far = far.reshape(m, n * per, pre)
            near = near.masked_fill(~seen[0], float("-inf"))
            top = far.amax(-1, keepdim=True)
            if longest:
                top = torch.maximum(top, near.amax(-1, keepdim=True))
            far, near = far.sub_(top).exp_(), near.sub_(top).exp_()
            total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
            y = torch.matmul(far.reshape(-1, pre), v[h]).reshape(m, n * per, dim) + torch.matmul(near, ov[h])
            y = torch.where(real[0], y / total, torch.zeros_like(y))
            z = torch.where(real[0], torch.log(total) + top, torch.full_like(top, float("-inf")))
            mine = slice(h * per, (h + 1) * per)
            out[lo:hi, :, mine] = y.reshape(m, n, per, dim).to(q.dtype)
            lse[lo:hi, :, mine] = z.reshape(m, n, per)
            del far, near
    return [out, lse]


# ---- sinks and shared: the definition in 64 bits ------------------------------------------------------------------

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


def _rows64(q, k, v, hidden):
    """One request and kv head: q [n, per, D], k and v [tokens, D], hidden [n, tokens]."""
    score = torch.einsum("iad,pd->aip", q, k) * q.shape[-1] ** -0.5
    score[:, hidden] = float("-inf")
    z = torch.logsumexp(score, -1)
    weight = torch.where(torch.isinf(z)[..., None], torch.zeros_like(score), torch.exp(score - z[..., None]))
    return torch.einsum("aip,pd->iad", weight, v), z.transpose(0, 1)


def _exact_attention(case, x, tokens):
    """tokens(b): positions that some query of request b may see, their keys and values."""
    q = x["q"].to(torch.float64)
    per = case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        before, new = int(x["before"][b]), int(x["new"][b])
        if new == 0 or int(x["count"][b]) == 0:
            continue
        pos, k, v = tokens(b)
        row = before + torch.arange(new, device="cuda")[:, None]
        hidden = pos > row
        if "window" in case:
            hidden = hidden | ((pos <= row - case["window"]) & (pos >= case["sinks"]))
        for h in range(case["kv_heads"]):
            mine = slice(h * per, (h + 1) * per)
            out[b, :new, mine], lse[b, :new, mine] = _rows64(q[b, :new, mine], k[:, h], v[:, h], hidden)
    return [out, lse]


def _exact_sinks(case, seed):
    x = _sinks_inputs(case, seed)

    def tokens(b):
        pos = torch.arange(int(x["count"][b]), device="cuda")
        pos = pos[(pos < case["sinks"]) | (pos > int(x["before"][b]) - case["window"])]
        return pos, _held(x["k"][b, pos]), _held(x["v"][b, pos])

    return _exact_attention(case, x, tokens)


def _exact_shared(case, seed):
    x = _shared_inputs(case, seed)
    last = [None, None, None]

    def tokens(b):
        g, pre, begin = int(x["group"][b]), int(x["pre"][x["group"][b]]), int(x["begin"][b])
        if last[0] != g:
            last[:] = g, _held(x["pk"][g, :pre]), _held(x["pv"][g, :pre])
        count = int(x["count"][b])
        k, v = (torch.cat([p, _held(x[name][b, pre - begin:count - begin])]) for p, name in ((last[1], "k"), (last[2], "v")))
        return torch.arange(count, device="cuda"), k, v

    return _exact_attention(case, x, tokens)


# ---- preparation and one pass -------------------------------------------------------------------------------------

def prepare(case, seed):
    """What a program has before the call: the pool's state, a projection's output, or the filled cache with its page
    table, lengths and queries.  A program that uses the plain form keeps the plain form of the cache."""
    s = dict(case=dict(case))
    if own:
        from speculative_decoding_verification_draft_gb300 import ssdv
        s["ssdv"] = ssdv
    if case["op"] == "plan":
        x = _plan_inputs(case, seed)
        s.update({k: _ints(x[k]) for k in ("length", "new", "held", "table", "stack", "free")}, n=x["n"])
        s["shared"] = _ints(np.full(case["batch"], case["shared"]))
        return s
    if case["op"] == "rope":
        s.update(_rope_inputs(case, seed))
        return s
    x = _sinks_inputs(case, seed) if case["op"] == "sinks" else _shared_inputs(case, seed)
    s.update(q=x["q"], table=x["table"], before=_ints(x["before"]), new=_ints(x["new"]))
    if case["op"] == "sinks":
        writes = [(x["table"], np.zeros(case["batch"]), x["count"], x["k"], x["v"])]
        s["longest"] = int(x["count"].max())
    else:
        first = torch.from_numpy(x["start"][:-1]).cuda()
        shared_full = x["pre"] // case["page"] * case["page"]
        writes = [(x["table"][first].contiguous(), np.zeros(case["groups"]), shared_full, x["pk"], x["pv"]),
                  (x["table"], x["begin"], x["count"] - x["begin"], x["k"], x["v"])]
        s["start"], s["prefix"] = _ints(x["start"]), _ints(x["pre"])
        # lengths that the program also has on the host
        s["cut"], s["pre"] = x["start"].tolist(), x["pre"].tolist()
        s["own"] = [int(x["own"][lo:hi].max()) for lo, hi in zip(s["cut"][:-1], s["cut"][1:])]
    if own:
        s["cache"] = s["ssdv"].make_kv_cache(x["pool"], case["kv_heads"], case["dim"], case["page"], device="cuda")
    else:
        s["cache"] = _plain_cache(case, x["pool"])
    for table, start, count, k, v in writes:
        if own:
            s["ssdv"].kv_append(s["cache"], table, _ints(start), k, v, n_new=_ints(count))
        else:
            _plain_write(case, s["cache"], table, _ints(start), _ints(count), k, v)
    return s


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "sinks": _plain_sinks, "shared": _plain_shared}[op](case, s)
    if op == "plan":
        return list(s["ssdv"].kv_plan(s["table"], s["held"], s["stack"], s["free"], s["length"], s["n"], case["page"],
                                      n_new=s["new"], n_shared=s["shared"]))
    if op == "rope":
        return list(s["ssdv"].qk_norm_rope(s["q"], s["k"], s["length"], q_weight=s["weight"][0], k_weight=s["weight"][1],
                                           inv_freq=s["freq"], eps=EPS, interleaved=case["interleaved"], n_new=s["new"]))
    if op == "sinks":
        return list(s["ssdv"].kv_attention(s["cache"], s["table"], s["before"], s["q"], n_q=s["new"],
                                           window=case["window"], sinks=case["sinks"], past_only=case["past_only"],
                                           return_lse=True))
    return list(s["ssdv"].kv_attention_shared(s["cache"], s["table"], s["before"], s["q"], s["start"], s["prefix"],
                                              n_q=s["new"], past_only=case["past_only"], return_lse=True))


def exact(case, seed):
    return {"plan": _exact_plan, "rope": _exact_rope, "sinks": _exact_sinks, "shared": _exact_shared}[case["op"]](case, seed)
