"""Several samples of each prompt, by greedy speculative decoding, with a two-layer target whose keys and values live in
the 4-bit cache: the pages that a prompt fills are shared by its samples.

A round: the draft proposes gamma tokens; kv_plan finds pages for them; queries and keys are normed and rotated by their
positions (qk_norm_rope) and written to the cache (kv_append); the first layer attends to the prompt once for all of its
samples (kv_attention_shared), the second to a window and the first tokens (kv_attention with sinks); verify accepts a
prefix.  When the samples have ended their pages go back to the stack.

    python examples/kv_samples.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from speculative_decoding_verification_draft_gb300 import ssdv  # noqa: E402

WINDOW, SINKS = 48, 4


class Target:
    """Embedding, two attention layers, output projection; the draft is the same without the attention."""

    def __init__(self, dtype, vocab=512, heads=8, kv_heads=2, dim=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.dtype, self.vocab, self.heads, self.kv_heads, self.dim = dtype, vocab, heads, kv_heads, dim
        d = heads * dim
        self.embed, self.wo = rand(vocab, d), rand(d, vocab) / d ** 0.5
        self.qkv = [rand(d, (heads + 2 * kv_heads) * dim) / d ** 0.5 for _ in range(2)]
        self.norms = [(1 + 0.2 * rand(dim), 1 + 0.2 * rand(dim)) for _ in range(2)]
        self.inv_freq = 10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))

    def rows(self, x, layer):
        """Queries, keys and values of states x [B, n, d], slices of one projection."""
        y = (x @ self.qkv[layer]).view(*x.shape[:2], -1, self.dim).to(self.dtype)
        return y.split((self.heads, self.kv_heads, self.kv_heads), dim=2)

    def write(self, x, layer, cache, table, kv_len, n_new=None):
        q, k, v = self.rows(x, layer)
        wq, wk = self.norms[layer]
        q, k = ssdv.qk_norm_rope(q, k, kv_len, wq, wk, self.inv_freq, n_new=n_new)
        ssdv.kv_append(cache, table, kv_len, k, v, n_new=n_new)
        return q


def _step(target, tokens, caches, table, kv_len, n_new, first):
    """Logits of `tokens` [B, n] behind kv_len; first(q): the first layer's attention."""
    x = target.embed[tokens]
    q = target.write(x, 0, caches[0], table, kv_len, n_new)
    h = x + first(q).float().reshape(x.shape)
    q = target.write(h, 1, caches[1], table, kv_len, n_new)
    a = ssdv.kv_attention(caches[1], table, kv_len, q, n_q=n_new, window=WINDOW, sinks=SINKS)
    return (h + a.float().reshape(x.shape)) @ target.wo


def run(prompts=3, samples=4, gamma=4, prompt=150, rounds=12, page=16, dtype=torch.bfloat16, seed=0):
    """Returns (tokens of each sample, kv_len, mean kept per round, worst margin, free pages at the end, pages): the margin
    says how far below the largest logit an emitted token's lies when its position is computed again from the cache."""
    target = Target(dtype, seed=seed)
    g = torch.Generator().manual_seed(seed)
    B = prompts * samples
    width = -(-(prompt + 1 + (rounds + 1) * (gamma + 1)) // page)
    pages = prompts * width + B * width
    caches = [ssdv.make_kv_cache(pages, target.kv_heads, target.dim, page) for _ in range(2)]
    stack, n_free = ssdv.make_kv_pool(pages)
    ints = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")

    # each prompt once, 32 tokens at a time, in pages of its own
    lengths = torch.randint(prompt // 2, prompt + 1, (prompts,), generator=g)
    ids = torch.randint(0, target.vocab, (prompts, prompt), generator=g)
    table, held = ints(torch.full((prompts, width), -1)), ints([0] * prompts)
    plan = (table, held, stack, n_free)
    for at in range(0, prompt, 32):
        n = min(32, prompt - at)
        kv_len, n_new = ints(lengths.clamp(max=at)), ints((lengths - at).clamp(0, n))
        ssdv.kv_plan(*plan, kv_len, n, page, n_new=n_new, out=plan)
        _step(target, ids[:, at:at + n].cuda(), caches, table, kv_len, n_new,
              lambda q: ssdv.kv_attention(caches[0], table, kv_len, q, n_q=n_new))

    # the samples: the prompt's full pages are shared; its last tokens are fed again with a token of the sample's own
    full = lengths // page * page
    group_start, shared_len = ints(torch.arange(prompts + 1) * samples), ints(full)
    n_shared = ints((full // page).repeat_interleave(samples))
    own_table, own_held = table.repeat_interleave(samples, 0), n_shared.clone()
    own_table = torch.where(torch.arange(width, device="cuda") < n_shared[:, None], own_table, -1).int().contiguous()
    state = (own_table, own_held, stack, n_free)
    kv_len = ints(full.repeat_interleave(samples))
    history = [ids[b // samples, :lengths[b // samples]].tolist() + [int(torch.randint(0, target.vocab, (1,), generator=g))]
               for b in range(B)]
    tail = [h[int(full[b // samples]):] for b, h in enumerate(history)]

    def attend(q, n_new=None):
        return ssdv.kv_attention_shared(caches[0], own_table, kv_len, q, group_start, shared_len, n_q=n_new)

    def feed(tokens, n_new=None):
        ssdv.kv_plan(*state, kv_len, tokens.shape[1], page, n_new=n_new, n_shared=n_shared, out=state)
        return _step(target, tokens, caches, own_table, kv_len, n_new, lambda q: attend(q, n_new))

    longest = max(map(len, tail)) - 1
    if longest:
        n_new = ints([len(t) - 1 for t in tail])
        feed(torch.tensor([t[:-1] + [0] * (longest + 1 - len(t)) for t in tail], device="cuda"), n_new)
        kv_len += n_new
    last = torch.tensor([h[-1] for h in history], device="cuda")
    begun = [len(h) for h in history]

    kept = 0
    for r in range(rounds):
        tokens = last[:, None]
        for i in range(gamma):
            tokens = torch.cat([tokens, (target.embed[tokens[:, -1]] @ target.wo).argmax(-1, keepdim=True)], 1)
        out, n = ssdv.verify(feed(tokens).float().contiguous(), None, tokens[:, 1:].int().contiguous(), temperature=0.0, seed=r)
        kv_len += n + 1
        last = out.long().gather(1, n.long()[:, None])[:, 0]
        for b, (row, m) in enumerate(zip(out.tolist(), n.tolist())):
            history[b] += row[: m + 1]
            kept += m + 1
    margin = max(_margin(target, caches, own_table[b:b + 1].contiguous(), history[b], begun[b]) for b in range(B))
    lens = kv_len.tolist()
    # all samples end, then the prompts
    ssdv.kv_plan(*state, ints([0] * B), 0, page, n_shared=n_shared, out=state)
    ssdv.kv_plan(*plan, ints([0] * prompts), 0, page, out=plan)
    if ssdv.read_status(ssdv.kv_workspace()):
        raise RuntimeError("the cache calls reported an error")
    return history, lens, kept / (rounds * B), margin, int(n_free), pages


def _margin(target, caches, table, tokens, begun):
    """The positions from begun - 1 on again, from the cache's values, in fp32 but for the roundings of the calls."""
    n = len(tokens) - 1  # the last token has not been fed yet
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = target.embed[torch.tensor(tokens[:n], device="cuda")][None]
    pos = torch.arange(n, device="cuda")
    angle = pos[:, None].double() * target.inv_freq.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    for layer in range(2):
        q = target.rows(x, layer)[0][0].float()
        q = q * (q.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * target.norms[layer][0]
        a, b = q.chunk(2, -1)
        q = torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(target.dtype).float()
        k, v = ssdv.kv_read(caches[layer], table, start, n, dtype=torch.float32)
        k, v = (t[0].repeat_interleave(target.heads // target.kv_heads, 1) for t in (k, v))
        hidden = pos[None] > pos[:, None]
        if layer == 1:
            hidden = hidden | ((pos[None] <= pos[:, None] - WINDOW) & (pos[None] >= SINKS))
        scores = torch.einsum("ihd,phd->hip", q, k) * target.dim ** -0.5
        y = torch.einsum("hip,phd->ihd", scores.masked_fill(hidden, float("-inf")).softmax(-1), v)
        x = x + y.to(target.dtype).float().reshape(1, n, -1)
    logits = (x @ target.wo)[0, begun - 1:]
    chosen = logits.gather(1, torch.tensor(tokens[begun:], device="cuda")[:, None])[:, 0]
    return float((logits.amax(1) - chosen).max())


if __name__ == "__main__":
    history, kv_len, kept, margin, free, pages = run()
    print(f"{kept:.2f} tokens kept a round; lengths {kv_len}; worst margin {margin:.4f}; {free} of {pages} pages free")
