"""Rounds of greedy speculative decoding with a one-layer target whose keys and values live in the 4-bit cache.

A round: the draft proposes gamma tokens; their keys and values, and the last token's, are written to the cache
(kv_append) behind kv_len; one attention call reads it for all gamma + 1 positions (kv_attention); verify accepts a
prefix and corrects the next token; kv_len moves by what was kept.  Rejected tokens need no undoing: the next round
writes over them.

    python examples/kv_round.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from speculative_decoding_verification_draft_gb300 import ssdv  # noqa: E402


class Layer:
    """Embedding, one attention layer, output projection; the draft is the same without the attention."""

    def __init__(self, vocab=512, heads=8, kv_heads=2, dim=64, longest=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.vocab, self.heads, self.kv_heads, self.dim = vocab, heads, kv_heads, dim
        d = heads * dim
        self.embed, self.place = rand(vocab, d), 0.3 * rand(longest, d)
        self.wq, self.wk, self.wv, self.wo = (rand(d, n) / d ** 0.5 for n in (d, kv_heads * dim, kv_heads * dim, vocab))

    def state(self, tokens, positions):
        return self.embed[tokens] + self.place[positions]

    def qkv(self, x):
        B, n = x.shape[:2]
        return ((x @ self.wq).view(B, n, self.heads, self.dim).bfloat16(),
                (x @ self.wk).view(B, n, self.kv_heads, self.dim).bfloat16(),
                (x @ self.wv).view(B, n, self.kv_heads, self.dim).bfloat16())

    def logits(self, x, attended=None):
        h = x if attended is None else x + attended.float().reshape(x.shape)
        return h @ self.wo


def run(batch=8, gamma=4, prompt=100, rounds=20, page_size=32, seed=0):
    """Returns (tokens of each request, kv_len, mean kept per round, worst margin): the margin says how far below the
    largest logit an emitted token's lies when its position is computed again from the cache, in fp32."""
    layer = Layer(seed=seed)
    g = torch.Generator().manual_seed(seed)
    longest = prompt + rounds * (gamma + 1) + gamma + 1
    per_request = -(-longest // page_size)
    cache = ssdv.make_kv_cache(batch * per_request, layer.kv_heads, layer.dim, page_size)
    table = torch.randperm(batch * per_request, generator=g).int().view(batch, per_request).cuda()

    # prompts of different lengths; the last token of each is fed with the first drafts
    lengths = torch.randint(1, prompt + 1, (batch,), generator=g)
    ids = torch.randint(0, layer.vocab, (batch, prompt + 1), generator=g)
    history = [ids[b, : lengths[b] + 1].tolist() for b in range(batch)]
    _, k, v = layer.qkv(layer.state(ids[:, :prompt].cuda(), torch.arange(prompt, device="cuda")))
    kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")
    ssdv.kv_append(cache, table, kv_len, k, v, n_new=lengths.int().cuda())
    kv_len += lengths.int().cuda()
    last = torch.tensor([h[-1] for h in history], device="cuda")

    kept = 0
    for r in range(rounds):
        tokens = last[:, None]
        for i in range(gamma):
            x = layer.state(tokens[:, -1], kv_len.long() + i)
            tokens = torch.cat([tokens, layer.logits(x).argmax(-1, keepdim=True)], 1)
        x = layer.state(tokens, kv_len.long()[:, None] + torch.arange(gamma + 1, device="cuda"))
        q, k, v = layer.qkv(x)
        ssdv.kv_append(cache, table, kv_len, k, v)
        target = layer.logits(x, ssdv.kv_attention(cache, table, kv_len, q))
        out, n = ssdv.verify(target, None, tokens[:, 1:].int().contiguous(), temperature=0.0, seed=r)
        kv_len += n + 1
        last = out.long().gather(1, n.long()[:, None])[:, 0]
        for b, (row, m) in enumerate(zip(out.tolist(), n.tolist())):
            history[b] += row[: m + 1]
            kept += m + 1
    if ssdv.read_status(ssdv.kv_workspace()):
        raise RuntimeError("the cache calls reported an error")
    return history, kv_len.tolist(), kept / (rounds * batch), _margin(layer, cache, table, history, lengths.tolist())


def _margin(layer, cache, table, history, lengths):
    worst = 0.0
    for b, tokens in enumerate(history):
        n = len(tokens) - 1  # the last token has not been fed yet
        start = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = ssdv.kv_read(cache, table[b:b + 1].contiguous(), start, n, dtype=torch.float32)
        x = layer.state(torch.tensor(tokens[:n], device="cuda"), torch.arange(n, device="cuda"))[None]
        q = layer.qkv(x)[0].float().transpose(1, 2)
        k, v = (t.transpose(1, 2).repeat_interleave(layer.heads // layer.kv_heads, 1) for t in (k, v))
        scores = (q @ k.transpose(2, 3) * layer.dim ** -0.5).masked_fill(
            torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
        logits = layer.logits(x, (scores.softmax(-1) @ v).transpose(1, 2))[0, lengths[b]:]
        chosen = logits.gather(1, torch.tensor(tokens[lengths[b] + 1:], device="cuda")[:, None])[:, 0]
        worst = max(worst, float((logits.amax(1) - chosen).max()))
    return worst


if __name__ == "__main__":
    history, kv_len, kept, margin = run()
    print(f"{kept:.2f} tokens kept a round; lengths {kv_len}; worst margin {margin:.4f}")
