"""Draft and verify with one attention layer: the attention block's operators
and those around it, next to the path selector, as a serving loop uses them.

A small random model (embedding, one attention layer with per-head norms,
rotation and grouped heads, tied output head) decodes several sequences in
blocks. Per step and sequence:

  1. the path selector drafts L tokens from hidden states of the block
     (here: embeddings of the tokens that usually follow one another, which
     the attention sometimes overrules);
  2. dflash_pages_extend gives the block its pages and places;
  3. the model runs over the last verified token and the drafts together:
     projection, dflash_paged_append (which also transforms the queries),
     dflash_paged_attend, output projection with the residual, output head
     (dflash_linear_run);
  4. dflash_logits_adjust takes the best tokens, with a penalty for tokens that
     have occurred if asked for, and dflash_verify_prefix keeps the accepted
     drafts and the next token;
  5. dflash_pages_trim moves the sequence's length back to what was kept, and
     takes back the pages of the rest. Rejected rows stay in the cache and are
     overwritten by the next append.

Greedy verification is lossless: the emitted tokens are those of decoding one
token at a time, which `check=True` (the default here) does as well, through
the same entry points with one new token per call. With sample=True the target's
probabilities decide instead, by rejection sampling.

    python examples/verify_block.py [--steps 24] [--fp8] [--repetition 1.3] [--sample]
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
        self.pool = pkg.PagePool.empty(requests=batch, cols=cols, num_pages=batch * cols, page_size=page)
        self.pool.free_pages.copy_(torch.randperm(batch * cols, device="cuda", generator=g))
        self.qkv = pkg.Linear(self.Wqkv)
        self.out = pkg.Linear(self.Wo, out_dtype=torch.float32)
        self.head = pkg.Linear(self.E, out_dtype=torch.float32)
        self.layer = pkg.PagedAttention(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page,
                                        dtype=torch.bfloat16, cache_dtype=kind, max_batch=batch)

    def hidden(self, tokens, batch):
        """Hidden states [tokens, d] of the batch's new tokens (flat), whose keys and values join the cache."""
        n = tokens.shape[0]
        qkv = self.qkv(self.E[tokens]).view(n, self.heads + 2 * self.kv_heads, self.head_dim)
        q = torch.empty(n, self.heads, self.head_dim, device="cuda", dtype=torch.bfloat16)
        self.layer.append(self.cache, batch, qkv[:, self.heads:self.heads + self.kv_heads], qkv[:, self.heads + self.kv_heads:],
                          self.transform, q=qkv[:, :self.heads], q_out=q)
        out = self.layer.attend(self.cache, batch, q)
        # a token's usual successor, unless what the attention finds in the context outweighs it
        return self.out(out.view(n, -1), residual=0.07 * self.E[self.follow(tokens)].float())

    def follow(self, tokens):
        return (tokens.long() * 7 + 1) % self.vocab

    def logits(self, tokens, batch):
        """fp32 logits [tokens, vocab] of the batch's new tokens."""
        return self.head(self.hidden(tokens, batch).to(torch.bfloat16))


class Answers:
    """The sequences so far, as the penalties take them."""

    def __init__(self, prompts, most, repetition):
        B, dev = len(prompts), "cuda"
        self.tokens = torch.zeros(B, most, device=dev, dtype=torch.int32)
        for b, p in enumerate(prompts):
            self.tokens[b, :len(p)] = p
        self.prompt_lens = torch.tensor([len(p) for p in prompts], device=dev, dtype=torch.int32)
        self.lens = self.prompt_lens.clone()
        penalties = {} if repetition == 1 else dict(repetition=torch.full((B,), repetition, device=dev),
                                                    presence=torch.full((B,), 0.5, device=dev))
        self.rules = pkg.LogitsRules(self.tokens, self.lens, self.prompt_lens, **penalties)

    def add(self, emitted, count):
        """The first count[b] of emitted [batch, n] join sequence b."""
        n = emitted.shape[1]
        at = (self.lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)).long()
        keep = torch.arange(n, device="cuda") < count[:, None]
        at = at.clamp(max=self.tokens.shape[1] - 1)
        self.tokens.scatter_(1, at, torch.where(keep, emitted, self.tokens.gather(1, at)))
        self.lens += count.to(torch.int32)


def decode(model, prompts, steps, L, repetition=1.0, sample=False, most=512):
    """Tokens that `steps` steps of L drafts emit for each prompt, and the mean accepted drafts per step."""
    B, dev = len(prompts), "cuda"
    V = model.vocab
    answers = Answers(prompts, most + (L + 1) * (steps + 1), repetition)
    cu, lens = torch.zeros(B + 1, device=dev, dtype=torch.int32), torch.zeros(B, device=dev, dtype=torch.int32)
    table = torch.zeros_like(model.pool.page_table)

    def extend(new):
        """The batch of a step with `new` more tokens for every sequence."""
        batch = pkg.PagedBatch(cu, lens, table, max_tokens=max(new))
        model.pool.extend(batch, torch.tensor(new, device=dev, dtype=torch.int32))
        return batch

    def best(logits, draft=None):
        target = torch.empty(logits.shape[:2], device=dev, dtype=torch.int32)
        pkg.dflash_logits_adjust(logits, answers.rules, argmax=target, draft=draft)
        return target
    logits = model.logits(torch.cat(prompts), extend([len(p) for p in prompts]))
    last = best(logits[cu[1:].long() - 1].view(B, 1, V)).view(-1)  # the prompts' next tokens: not yet in the cache
    one = torch.ones(B, device=dev, dtype=torch.int32)
    answers.add(last[:, None], one)
    done = [[int(t)] for t in last]
    if L == 0:                                           # one token at a time
        for _ in range(steps):
            last = best(model.logits(last, extend([1] * B)).view(B, 1, V)).view(-1)
            answers.add(last[:, None], one)
            for b in range(B):
                done[b].append(int(last[b]))
        return done, 0.0
    W = model.E
    g = torch.Generator(device=dev).manual_seed(1)
    WA, WB, WH = ((model.d ** -0.5 * torch.randn(256, model.d, device=dev, generator=g)).to(torch.bfloat16) for _ in range(3))
    accept, emitted = torch.empty(B, device=dev, dtype=torch.int32), torch.empty(B, L + 1, device=dev, dtype=torch.int32)
    probs = torch.empty(B, L + 1, V, device=dev) if sample else None
    kept = 0
    walk = pkg.DFLASH_WALK_SAMPLE if sample else pkg.DFLASH_WALK_VITERBI
    with pkg.Selector(W, W, WA, WB, WH, L=L, K=16, max_batch=B, walk=walk) as selector:
        for _ in range(steps):
            guess = [model.follow(last)]
            while len(guess) < L:
                guess.append(model.follow(guess[-1]))
            hidden = 4 * W[torch.stack(guess, 1)]
            if sample:
                out = selector.outputs(B)
                q = torch.empty(B, L, 16, device=dev)
                pkg.dflash_select_run_sampled(selector.h, hidden, last, torch.rand(B, L, device=dev, generator=g), draft_probs=q, **out)
                draft = out["path"]
            else:
                draft = selector.run(hidden, last)["path"]
            tokens = torch.cat([last[:, None], draft], 1).view(-1)
            logits = model.logits(tokens, extend([L + 1] * B)).view(B, L + 1, V)
            if sample:
                pkg.dflash_logits_adjust(logits, answers.rules, probs=probs, draft=draft)
                pkg.dflash_verify_rejection(draft, out["topk_ids"], q, probs, torch.rand(B, L, device=dev, generator=g),
                                            torch.rand(B, device=dev, generator=g), accept, emitted)
            else:
                pkg.dflash_verify_prefix(draft, best(logits, draft), accept, emitted)
            model.pool.trim(accepted=accept, drafts=L)   # what was accepted stays
            answers.add(emitted, accept + 1)
            last = emitted.gather(1, accept[:, None].long()).view(-1)
            for b, n in enumerate(accept.tolist()):
                done[b] += emitted[b, :n + 1].tolist()
                kept += n
        pkg.dflash_select_sync_status(selector.h)
    model.layer.sync_status()
    for layer in (model.qkv, model.out, model.head):
        layer.sync_status()
    return done, kept / (steps * B)


def main(steps=24, L=7, fp8=False, check=True, seed=0, repetition=1.0, sample=False):
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(0, 2048, (n,), generator=g, dtype=torch.int32).cuda() for n in (5, 33, 70)]
    blocks, mean = decode(Model(fp8=fp8, seed=seed), prompts, steps, L, repetition, sample)
    print(f"{steps} steps of {L} drafts: {[len(t) for t in blocks]} tokens, {mean:.2f} drafts accepted per step")
    if check and not sample:
        single, _ = decode(Model(fp8=fp8, seed=seed), prompts, max(map(len, blocks)), 0, repetition)
        same = [sum(a == b for a, b in zip(x, y)) for x, y in zip(blocks, single)]
        print(f"tokens equal to decoding one at a time: {same} of {[len(t) for t in blocks]}")
        return blocks, single
    return blocks, None


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--fp8", action="store_true", help="an 8-bit cache")
    ap.add_argument("--repetition", type=float, default=1.0, help="penalty for tokens that have occurred")
    ap.add_argument("--sample", action="store_true", help="rejection sampling instead of greedy verification")
    a = ap.parse_args()
    main(steps=a.steps, fp8=a.fp8, repetition=a.repetition, sample=a.sample)
