"""A rollout whose numbers do not depend on the batch, and a training step on it.

A small decoder-only model, tensor-parallel over P ranks held as P sets of
buffers on one GPU: each rank has its own heads, its own paged key-value cache
and its own slice of the vocabulary.  Every decoding step

* appends the new token's keys and values to each rank's cache, rotating
  queries and keys to their position (``kv_append``),
* attends over the cache (``paged_attention``),
* adds the ranks' partial projections in a fixed order (``all_reduce``), and
* scores the vocabulary shards without gathering them (``token_logprobs``),
  which also gives the next greedy token.

Because each of these gives a sequence the same bits whatever else is in the
call, a sequence rolled out alone and in a batch has the same tokens and the
same log probabilities, bit for bit.  ``train_step`` then scores the rollout's
tokens again, with the gradient of a policy loss and an entropy bonus with
respect to the head's shards (``logprobs_and_entropy``), and starts from
exactly the log probabilities that the rollout recorded.

    python examples/reproducible_rollout.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import reduce_copy_rank_gb300 as dc  # noqa: E402

ROWS = 16  # every product has this many rows (a batch is padded to it), so that a row's product is one fixed kernel


class Model:
    """Random weights of a small decoder, split over `ranks` ranks."""

    def __init__(self, ranks=2, layers=2, hidden=512, heads=8, kv_heads=2, dim=64, vocab=4099, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.ranks, self.dim, self.vocab, self.device = ranks, dim, vocab, device
        self.q_heads, self.kv_heads = heads // ranks, kv_heads // ranks  # of one rank
        self.embedding = weight(vocab, hidden) * hidden ** 0.5
        per = self.q_heads + 2 * self.kv_heads
        self.qkv = [[weight(per * dim, hidden) for _ in range(ranks)] for _ in range(layers)]
        self.out = [[weight(hidden, self.q_heads * dim) for _ in range(ranks)] for _ in range(layers)]
        bounds = [vocab * r // ranks for r in range(ranks + 1)]
        self.head = [weight(b - a, hidden) * 4 for a, b in zip(bounds, bounds[1:])]
        angle = torch.arange(4096, device=device, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()


class Cache:
    """Each layer's and rank's paged cache, one page table for all of them."""

    def __init__(self, model: Model, sequences: int, tokens: int, page: int = 16):
        per = -(-tokens // page)
        shape = (sequences * per, page, model.kv_heads, model.dim)
        self.k, self.v = ([[torch.empty(shape, device=model.device, dtype=torch.bfloat16) for _ in range(model.ranks)]
                           for _ in model.qkv] for _ in range(2))
        self.table = torch.randperm(sequences * per, device=model.device).to(torch.int32).view(sequences, per)
        self.lengths = torch.zeros(sequences, device=model.device, dtype=torch.int32)
        self.seqs = torch.arange(sequences, device=model.device, dtype=torch.int32)
        self.workspace = dc.attention_workspace(sequences, model.q_heads, model.kv_heads, model.dim, per * page,
                                                model.device)


def norm(x):
    """Root-mean-square norm of bfloat16 rows, in binary32."""
    y = x.float()
    return (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def project(x, w):
    """x @ w.T with the rows padded to ROWS."""
    full = torch.zeros(ROWS, x.shape[1], device=x.device, dtype=x.dtype)
    full[:len(x)] = x
    return (full @ w.t())[:len(x)]


def step(model: Model, cache: Cache, tokens):
    """One token of every sequence through the model: the last hidden rows."""
    n, hq, hk, d = len(tokens), model.q_heads, model.kv_heads, model.dim
    x = model.embedding[tokens]
    positions = cache.lengths.clone()
    cache.lengths += 1
    for layer, (qkv, out) in enumerate(zip(model.qkv, model.out)):
        y = norm(x)
        partial = []
        for r in range(model.ranks):
            both = project(y, qkv[r]).view(n, hq + 2 * hk, d)
            q = torch.empty(n, hq, d, device=x.device, dtype=x.dtype)
            dc.kv_append(both[:, hq:hq + hk], both[:, hq + hk:], positions, cache.seqs, cache.table, cache.k[layer][r],
                         cache.v[layer][r], q=both[:, :hq], q_out=q, cos_sin=model.cos_sin)
            attended = dc.paged_attention(q, cache.k[layer][r], cache.v[layer][r], cache.table, cache.lengths,
                                          torch.empty_like(q), cache.workspace)
            partial.append(project(attended.view(n, -1), out[r]).contiguous())
        sums = [torch.empty_like(p) for p in partial]
        x = x + dc.all_reduce(partial, sums, order="tree")[0]
    return norm(x)


def rollout(model: Model, prompts, new_tokens: int):
    """Greedy continuations of `prompts` (int64 [sequences, prompt tokens], at
    most ROWS sequences): the tokens, their log probabilities and the hidden
    rows that chose them, each [new_tokens, sequences, ...]."""
    n, prompt = prompts.shape
    cache = Cache(model, n, prompt + new_tokens)
    for i in range(prompt):
        hidden = step(model, cache, prompts[:, i])
    tokens, logprobs, rows = [], [], []
    for i in range(new_tokens):
        shards = [project(hidden, w) for w in model.head]
        best = torch.empty(n, 1, device=model.device)
        token = torch.empty(n, 1, device=model.device, dtype=torch.int64)
        lp = torch.empty(n, device=model.device)
        # (no token to score yet: -1)
        dc.token_logprobs(shards, torch.full((n,), -1, device=model.device), lp, top_logprobs=best, top_tokens=token)
        tokens.append(token[:, 0])
        logprobs.append(best[:, 0])
        rows.append(hidden)
        if i + 1 < new_tokens:
            hidden = step(model, cache, token[:, 0])
    return torch.stack(tokens), torch.stack(logprobs), torch.stack(rows)


def train_step(model: Model, tokens, hidden, advantages, entropy_bonus=0.01):
    """Log probabilities of a rollout's tokens and the gradient of the policy
    loss -(advantage * log probability + bonus * entropy) with respect to the
    head's shards."""
    weights = [w.detach().clone().requires_grad_() for w in model.head]
    logprobs, loss = [], 0.0
    for t, h, a in zip(tokens, hidden, advantages):
        lp, entropy = dc.logprobs_and_entropy([project(h, w) for w in weights], t)
        loss = loss - (a * lp).sum() - entropy_bonus * entropy.sum()
        logprobs.append(lp.detach())
    loss.backward()
    return torch.stack(logprobs), [w.grad for w in weights]


def main():
    model = Model()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(0, model.vocab, (5, 12), generator=g, device="cuda")
    tokens, logprobs, hidden = rollout(model, prompts, 24)
    same = True
    for b in range(len(prompts)):
        t, lp, _ = rollout(model, prompts[b:b + 1], 24)
        same &= torch.equal(t[:, 0], tokens[:, b]) and torch.equal(lp[:, 0], logprobs[:, b])
    print(f"5 sequences of 12 + 24 tokens: alone and together the same bits: {same}")
    advantages = torch.randn(tokens.shape, generator=g, device="cuda")
    scored, grads = train_step(model, tokens, hidden, advantages)
    print(f"training scores equal the rollout's: {torch.equal(scored, logprobs)}; "
          f"gradient norm {float(sum(x.float().square().sum() for x in grads)) ** 0.5:.4f}")
    return 0 if same and torch.equal(scored, logprobs) else 1


if __name__ == "__main__":
    sys.exit(main())
