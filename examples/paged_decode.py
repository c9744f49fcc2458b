"""Tree-speculative decoding over the paged 4-bit cache, end to end.

A toy target (random attention layers over a token embedding, no MLP) decodes a
batch of prompts of different lengths.  Each step

  1. drafts a tree of tokens per request (DDTree over toy marginals),
  2. makes room for its nodes (cache_reserve) and, layer by layer, writes their
     keys and values behind the context (cache_append) and attends under the
     ancestor masks (cache_attend),
  3. walks the tree along the target's choices (verify_tree),
  4. keeps the accepted path's rows (cache_compact) and gives back the pages
     that the rest took (cache_release).

Half way every request is forked (cache_fork): the copies share full pages and
must go on with the same tokens.  Greedy tree verification commits what plain
greedy decoding commits, so the example decodes once more a token at a time and
compares.

    python examples/paged_decode.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import speculative_decoding_draft_sampling_gb300 as sv  # noqa: E402


class Target:
    """Attention layers with residuals over a token embedding; logits by a scaled
    output matrix (well separated, so that choices do not hang on rounding)."""

    def __init__(self, vocab=512, layers=2, q_heads=8, kv_heads=2, head_dim=64, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        width = q_heads * head_dim

        def mat(*shape, scale):
            return (scale * torch.randn(shape, device=device, generator=g)).to(torch.bfloat16)

        self.vocab, self.layers, self.hq, self.hkv, self.d = vocab, layers, q_heads, kv_heads, head_dim
        self.embed = mat(vocab, width, scale=1.0)
        self.position = mat(64, width, scale=0.5)
        self.qkv = [mat(width, (q_heads + 2 * kv_heads) * head_dim, scale=1 / math.sqrt(width)) for _ in range(layers)]
        self.out = [mat(width, width, scale=1 / math.sqrt(width)) for _ in range(layers)]
        self.head = mat(width, vocab, scale=8 / math.sqrt(width))

    def rows(self, tokens, positions):
        return self.embed[tokens.long().clamp(min=0)] + self.position[positions % 64]

    def forward(self, tokens, positions, cache, ctx, rows, mask=None, depth=None):
        """Logits [B, n, vocab] fp32 of drafted rows, whose K and V go into the cache at ctx."""
        x = self.rows(tokens, positions)
        B, n = tokens.shape
        split = [self.hq * self.d, self.hkv * self.d, self.hkv * self.d]
        for layer in range(self.layers):
            q, k, v = (x @ self.qkv[layer]).split(split, -1)
            pool = cache.pool[layer]
            sv.cache_append(k.unflatten(-1, (self.hkv, self.d)), v.unflatten(-1, (self.hkv, self.d)), pool,
                            cache.pages.page_table, ctx, rows, status=cache.status)
            a = sv.cache_attend(q.unflatten(-1, (self.hq, self.d)), pool, cache.pages.page_table, ctx, rows,
                                anc_mask=mask, depth=depth, status=cache.status)
            x = x + a.out.flatten(2) @ self.out[layer]
        return (x @ self.head).float()


class Cache:
    """The pools of all layers and who holds which page."""

    def __init__(self, target, requests, max_tokens, page_size=16, device="cuda"):
        self.page, self.d = page_size, target.d
        per = -(-max_tokens // page_size)
        self.pages = sv.page_state(requests, per, requests * per, device)
        self.pool = torch.zeros((target.layers, requests * per, target.hkv, sv.cache_block_bytes(target.d, page_size)),
                                dtype=torch.uint8, device=device)
        self.status = torch.zeros(requests, dtype=torch.int32, device=device)


def prefill(target, cache, prompts, lengths):
    """All but the last token of each prompt into the cache; what is left is decoding's first root."""
    n = prompts.shape[1]
    pos = torch.arange(n, device=prompts.device).expand_as(prompts)
    sv.cache_reserve(cache.pages, lengths, cache.page, status=cache.status)
    target.forward(prompts, pos, cache, torch.zeros_like(lengths), lengths - 1)
    return lengths - 1, prompts.gather(1, (lengths - 1).long()[:, None])[:, 0]


def step_greedy(target, cache, ctx, root):
    """One token a step."""
    one = torch.ones_like(ctx)
    sv.cache_reserve(cache.pages, ctx + 1, cache.page, status=cache.status)
    logits = target.forward(root[:, None], ctx[:, None].long(), cache, ctx, one)
    return ctx + 1, logits[:, 0].argmax(-1).to(torch.int32)


def draft(target, root, ctx, depth, gen):
    """Toy marginals of the next `depth` tokens: the target's own continuation without its context, and noise."""
    q = []
    token = root
    for i in range(depth):
        logits = target.rows(token.long(), ctx.long() + i) @ target.head
        logits = logits.float() + 2.0 * torch.randn(logits.shape, device=logits.device, generator=gen)
        q.append(torch.softmax(logits, -1))
        token = logits.argmax(-1).to(torch.int32)
    return torch.stack(q, 1).contiguous()


def step_tree(target, cache, ctx, root, budget, depth, gen):
    """One draft tree a step: returns the new context, the next root and the committed tokens (-1 padded)."""
    tree = sv.tree_build(draft(target, root, ctx, depth, gen), budget)
    tokens = tree.token.clone()
    tokens[:, 0] = root
    sv.cache_reserve(cache.pages, ctx + tree.num_nodes, cache.page, status=cache.status)
    positions = ctx[:, None].long() + tree.depth.clamp(min=0).long()
    logits = target.forward(tokens, positions, cache, ctx, tree.num_nodes, tree.anc_mask, tree.depth)
    walk = sv.verify_tree(logits, tree.token, tree.parent, tree.num_nodes, depth)
    sv.cache_compact(cache.pool, cache.pages.page_table, ctx, walk.path_nodes, walk.num_accepted, cache.d,
                     status=cache.status)
    ctx = ctx + walk.num_accepted + 1
    sv.cache_release(cache.pages, ctx, cache.page, status=cache.status)
    root = walk.tokens.gather(1, walk.num_accepted.long()[:, None])[:, 0]
    return ctx, root, walk.tokens


def run(steps=8, requests=3, budget=24, depth=5, seed=0, device="cuda"):
    """Decodes by trees and a token at a time; returns both token lists per request and the accepted lengths."""
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    target = Target(seed=seed, device=device)
    longest = 40
    lengths = torch.tensor([longest - 13 * b % 37 for b in range(requests)], dtype=torch.int32, device=device)
    prompts = torch.randint(0, target.vocab, (requests, longest), generator=gen, device=device)
    room = longest + steps * (depth + 2) + budget + 16

    cache = Cache(target, 2 * requests, room, device=device)
    both = torch.arange(2 * requests, device=device)
    pad = torch.zeros(requests, dtype=torch.int32, device=device)
    ctx, root = prefill(target, cache, torch.cat([prompts, prompts]), torch.cat([lengths, pad + 1]))
    # the second half of the requests is idle until the first is forked into it
    sv.cache_release(cache.pages, torch.where(both < requests, ctx, 0).to(torch.int32), cache.page)
    ctx = torch.where(both < requests, ctx, 0).to(torch.int32)
    got, kept = [[] for _ in range(2 * requests)], []
    for i in range(steps):
        if i == steps // 2:
            src = torch.arange(requests, dtype=torch.int32, device=device)
            sv.cache_release(cache.pages, torch.where(both < requests, ctx, 0).to(torch.int32), cache.page)
            sv.cache_fork(cache.pool, cache.pages, src, src + requests, ctx, cache.d)
            ctx[requests:] = ctx[:requests]
            root[requests:] = root[:requests]
            got[requests:] = [list(t) for t in got[:requests]]
        ctx, root, tokens = step_tree(target, cache, ctx, root.to(torch.int32), budget, depth, gen)
        for b, row in enumerate(tokens.tolist()):
            got[b] += [t for t in row if t >= 0]
        kept.append(int((tokens >= 0).sum(1)[:requests].sum()))

    plain = Cache(target, requests, room, device=device)
    ctx, root = prefill(target, plain, prompts, lengths)
    want = [[] for _ in range(requests)]
    for _ in range(max(len(t) for t in got[:requests])):
        ctx, root = step_greedy(target, plain, ctx, root.to(torch.int32))
        for b, t in enumerate(root.tolist()):
            want[b].append(t)
    problems = int(cache.status.abs().sum() + plain.status.abs().sum())
    return got, want, kept, problems


if __name__ == "__main__":
    sv.build()
    got, want, kept, problems = run()
    half = len(got) // 2
    for b in range(half):
        n = len(got[b])
        print(f"request {b}: {n} tokens in {len(kept)} steps, the same as token by token: {got[b] == want[b][:n]}")
    print("forked requests agree:", all(g[:len(w)] == w[:len(g)] for g, w in zip(got[half:], want)))
    print("tokens committed a step:", kept, " status bits:", problems)
