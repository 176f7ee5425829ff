"""Draft and verify with one attention layer: the attention block's operators
next to the path selector, as a serving loop uses them.

A small random model (embedding, one attention layer with per-head norms,
rotation and grouped heads, tied output head) decodes several sequences in
blocks. Per step and sequence:

  1. the path selector drafts L tokens from hidden states of the block
     (here: embeddings of the tokens that usually follow one another, which
     the attention sometimes overrules);
  2. the model runs over the last verified token and the drafts together:
     projection, dflash_paged_append (which also transforms the queries),
     dflash_paged_attend, output head;
  3. dflash_verify_prefix keeps the accepted drafts and the next token;
  4. the sequence's length moves back to what was kept. Rejected rows stay in
     the cache and are overwritten by the next append.

Greedy verification is lossless: the emitted tokens are those of decoding one
token at a time, which `check=True` (the default here) does as well, through
the same entry points with one new token per call.

    python examples/verify_block.py [--steps 24] [--fp8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import speculative_decoding_draft_tcgen05_gb300 as pkg  # noqa: E402


class Model:
    """Random weights of one attention layer; keys and values in pages."""

    def __init__(self, vocab=2048, d=512, heads=8, kv_heads=2, head_dim=64, batch=3, most=512, page=16, fp8=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, std):
            return (std * torch.randn(*shape, device="cuda", generator=g)).to(torch.bfloat16)
        self.E = w(vocab, d, std=1.0)
        self.Wqkv = w((heads + 2 * kv_heads) * head_dim, d, std=d ** -0.5)
        self.Wo = w(d, heads * head_dim, std=2 * (heads * head_dim) ** -0.5)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * inv
        self.transform = pkg.QkTransform(torch.cat([angle.cos(), angle.sin()], 1).float(), q_weight=w(head_dim, std=0.1) + 1,
                                         k_weight=w(head_dim, std=0.1) + 1)
        self.heads, self.kv_heads, self.head_dim, self.d, self.vocab = heads, kv_heads, head_dim, d, vocab
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        cols = -(-most // page)
        shape = (batch * cols, page, kv_heads, head_dim)
        self.k, self.v = (torch.zeros(shape, device="cuda", dtype=torch.bfloat16).to(kind) for _ in range(2))
        self.cache = pkg.PagedCache(self.k, self.v, **(dict(k_scale=1 / 64, v_scale=1 / 64) if fp8 else {}))
        self.table = torch.randperm(batch * cols, device="cuda", generator=g).to(torch.int32).view(batch, cols)
        self.layer = pkg.PagedAttention(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page,
                                        dtype=torch.bfloat16, cache_dtype=kind, max_batch=batch)

    def hidden(self, tokens, batch):
        """Hidden states [tokens, d] of the batch's new tokens (flat), whose keys and values join the cache."""
        n = tokens.shape[0]
        qkv = (self.E[tokens] @ self.Wqkv.T).view(n, self.heads + 2 * self.kv_heads, self.head_dim)
        q = torch.empty(n, self.heads, self.head_dim, device="cuda", dtype=torch.bfloat16)
        self.layer.append(self.cache, batch, qkv[:, self.heads:self.heads + self.kv_heads], qkv[:, self.heads + self.kv_heads:],
                          self.transform, q=qkv[:, :self.heads], q_out=q)
        out = self.layer.attend(self.cache, batch, q)
        # a token's usual successor, unless what the attention finds in the context outweighs it
        return 0.07 * self.E[self.follow(tokens)].float() + out.view(n, -1).float() @ self.Wo.float().T

    def follow(self, tokens):
        return (tokens.long() * 7 + 1) % self.vocab

    def next_tokens(self, tokens, batch):
        return (self.hidden(tokens, batch) @ self.E.float().T).argmax(-1).to(torch.int32)


def decode(model, prompts, steps, L):
    """Tokens that `steps` steps of L drafts emit for each prompt, and the mean accepted drafts per step."""
    B, dev = len(prompts), "cuda"
    lens = torch.tensor([len(p) for p in prompts], device=dev, dtype=torch.int32)
    cu = torch.tensor([sum(len(p) for p in prompts[:i]) for i in range(B + 1)], device=dev, dtype=torch.int32)
    last = model.next_tokens(torch.cat(prompts), pkg.PagedBatch(cu, lens, model.table, max_tokens=max(map(len, prompts))))
    last = last[cu[1:].long() - 1]                       # the prompts' next tokens: emitted, not yet in the cache
    done = [[int(t)] for t in last]
    if L == 0:                                           # one token at a time
        one = pkg.PagedBatch(torch.arange(B + 1, device=dev, dtype=torch.int32), lens, model.table, max_tokens=1)
        for _ in range(steps):
            lens += 1
            last = model.next_tokens(last, one)
            for b in range(B):
                done[b].append(int(last[b]))
        return done, 0.0
    W = model.E
    g = torch.Generator(device=dev).manual_seed(1)
    WA, WB, WH = ((model.d ** -0.5 * torch.randn(256, model.d, device=dev, generator=g)).to(torch.bfloat16) for _ in range(3))
    cu = torch.arange(B + 1, device=dev, dtype=torch.int32) * (L + 1)
    block = pkg.PagedBatch(cu, lens, model.table, max_tokens=L + 1)
    accept, emitted = torch.empty(B, device=dev, dtype=torch.int32), torch.empty(B, L + 1, device=dev, dtype=torch.int32)
    kept = 0
    with pkg.Selector(W, W, WA, WB, WH, L=L, K=16, max_batch=B) as selector:
        for _ in range(steps):
            guess = [model.follow(last)]
            while len(guess) < L:
                guess.append(model.follow(guess[-1]))
            draft = selector.run(4 * W[torch.stack(guess, 1)], last)["path"]
            tokens = torch.cat([last[:, None], draft], 1).view(-1)
            lens += L + 1                                # the block's places
            target = model.next_tokens(tokens, block).view(B, L + 1)
            pkg.dflash_verify_prefix(draft, target, accept, emitted)
            lens -= L - accept                           # what was accepted stays
            last = emitted.gather(1, accept[:, None].long()).view(-1)
            for b, n in enumerate(accept.tolist()):
                done[b] += emitted[b, :n + 1].tolist()
                kept += n
        pkg.dflash_select_sync_status(selector.h)
    model.layer.sync_status()
    return done, kept / (steps * B)


def main(steps=24, L=7, fp8=False, check=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(0, 2048, (n,), generator=g).cuda() for n in (5, 33, 70)]
    blocks, mean = decode(Model(fp8=fp8, seed=seed), prompts, steps, L)
    print(f"{steps} steps of {L} drafts: {[len(t) for t in blocks]} tokens, {mean:.2f} drafts accepted per step")
    if check:
        single, _ = decode(Model(fp8=fp8, seed=seed), prompts, max(map(len, blocks)), 0)
        same = [sum(a == b for a, b in zip(x, y)) for x, y in zip(blocks, single)]
        print(f"tokens equal to decoding one at a time: {same} of {[len(t) for t in blocks]}")
        return blocks, single
    return blocks, None


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--fp8", action="store_true", help="an 8-bit cache")
    a = ap.parse_args()
    main(steps=a.steps, fp8=a.fp8)
