"""Several samples of each prompt behind its one cached copy, and a training step on them.

The decoder of ``reproducible_rollout`` with queries and keys normed per head.
A prompt goes through the model once, into pages that all of its samples share;
every decoding step of the samples then

* norms and rotates the new tokens' queries and keys on their way into each
  rank's cache (``kv_append`` with ``q_norm`` and ``k_norm``),
* attends to the shared prompt and to the sample's own tokens under one softmax,
  the prompt's keys and values read once for its samples (``prefix_attention``),
* draws a token by given random numbers, and records its log probability from
  the hidden row and the head's shards, without their logits
  (``linear_logprobs``).

A sample has the same bits alone and among others.  ``train_step`` scores the
samples' hidden rows again, all at once, and takes the gradient of a policy loss
with respect to those rows and to the head (``linear_logprobs_and_entropy``);
``attention_step`` takes a layer's normed queries and keys of whole sequences
with the gradient of the norms' weights (``normed_queries_and_keys``).

    python examples/group_rollout.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import reduce_copy_rank_gb300 as dc  # noqa: E402
from reproducible_rollout import Model, norm, project  # noqa: E402


class NormedModel(Model):
    """Model with weights that norm each layer's and rank's queries and keys."""

    def __init__(self, seed=0, **kw):
        super().__init__(seed=seed, **kw)
        g = torch.Generator(device=self.device).manual_seed(seed + 1)
        self.norms = [[[(1 + 0.2 * torch.randn(self.dim, generator=g, device=self.device)).to(torch.bfloat16) for _ in range(2)]
                       for _ in range(self.ranks)] for _ in self.qkv]


class Samples:
    """Caches of `each` samples of every prompt, one pool of pages a layer and rank.  Prompts fill whole pages: a
    sample's row of the table is its prompt's pages, then its own, and one position means one place to ``kv_append``."""

    def __init__(self, model, prompts: int, prompt_tokens: int, each: int, new_tokens: int, page: int = 16):
        if prompt_tokens % page:
            raise ValueError(f"prompts of {prompt_tokens} tokens do not fill pages of {page}")
        self.model, self.prompts, self.each, n = model, prompts, each, prompts * each
        wide, own = prompt_tokens // page, -(-new_tokens // page)
        shape = (prompts * wide + n * own, page, model.kv_heads, model.dim)
        self.k, self.v = ([[torch.empty(shape, device=model.device, dtype=torch.bfloat16) for _ in range(model.ranks)]
                           for _ in model.qkv] for _ in range(2))
        pages = torch.randperm(shape[0], device=model.device).to(torch.int32)
        self.prefix = pages[:prompts * wide].view(prompts, wide)
        self.table = torch.cat([self.prefix.repeat_interleave(each, 0), pages[prompts * wide:].view(n, own)], 1)
        self.own = self.table[:, wide:]
        self.prefix_lengths = torch.zeros(prompts, device=model.device, dtype=torch.int32)
        self.lengths = torch.zeros(n, device=model.device, dtype=torch.int32)  # of the samples' own tokens
        heads = model.q_heads, model.kv_heads, model.dim
        self.prompt_workspace = dc.attention_workspace(prompts, *heads, wide * page, model.device)
        self.workspace = dc.prefix_attention_workspace(n, prompts, *heads, wide * page, own * page, model.device)

    def step(self, tokens, prompt: bool):
        """One token of every prompt, or of every sample, through the model: the last hidden rows."""
        model, n = self.model, len(tokens)
        hq, hk, d = model.q_heads, model.kv_heads, model.dim
        x = model.embedding[tokens]
        if prompt:
            positions, table = self.prefix_lengths.clone(), self.prefix
            self.prefix_lengths += 1
        else:
            positions, table = self.prefix_lengths.repeat_interleave(self.each) + self.lengths, self.table
            self.lengths += 1
        seqs = torch.arange(n, device=x.device, dtype=torch.int32)
        for layer, (qkv, out) in enumerate(zip(model.qkv, model.out)):
            y = norm(x)
            partial = []
            for r in range(model.ranks):
                both = project(y, qkv[r]).view(n, hq + 2 * hk, d)
                q = torch.empty(n, hq, d, device=x.device, dtype=x.dtype)
                k, v, (q_norm, k_norm) = self.k[layer][r], self.v[layer][r], model.norms[layer][r]
                dc.kv_append(both[:, hq:hq + hk], both[:, hq + hk:], positions, seqs, table, k, v, q=both[:, :hq], q_out=q,
                             cos_sin=model.cos_sin, q_norm=q_norm, k_norm=k_norm)
                attended = torch.empty_like(q)
                if prompt:
                    dc.paged_attention(q, k, v, table, self.prefix_lengths, attended, self.prompt_workspace)
                else:
                    dc.prefix_attention(q, k, v, self.prefix, self.prefix_lengths, self.own, self.lengths, attended, self.workspace)
                partial.append(project(attended.view(n, -1), out[r]).contiguous())
            sums = [torch.empty_like(p) for p in partial]
            x = x + dc.all_reduce(partial, sums, order="tree")[0]
        return norm(x)


def rollout(model, prompts, each: int, noise):
    """`each` samples of every prompt (int64 [prompts, tokens]), drawn by adding `noise` ([new tokens, samples,
    vocabulary], Gumbel numbers) to the logits: the tokens, their log probabilities and the hidden rows that chose them,
    each [new tokens, samples, ...], and the caches."""
    n = len(prompts) * each
    cache = Samples(model, *prompts.shape, each, len(noise))
    for i in range(prompts.shape[1]):
        hidden = cache.step(prompts[:, i], prompt=True)
    hidden = hidden.repeat_interleave(each, 0)
    workspace = dc.linear_logprobs_workspace(n, hidden.shape[1], model.vocab, device=model.device)
    tokens, logprobs, rows = [], [], []
    for i, z in enumerate(noise):
        token = (torch.cat([project(hidden, w) for w in model.head], 1).float() + z).argmax(1)
        lp = torch.empty(n, device=model.device)
        dc.linear_logprobs(hidden, model.head, token, lp, workspace)
        tokens.append(token)
        logprobs.append(lp)
        rows.append(hidden)
        if i + 1 < len(noise):
            hidden = cache.step(token, prompt=False)
    return torch.stack(tokens), torch.stack(logprobs), torch.stack(rows), cache


def train_step(model, tokens, hidden, advantages, entropy_bonus=0.01):
    """Log probabilities of the samples' tokens and the gradient of the policy loss -(advantage * log probability +
    bonus * entropy) with respect to their hidden rows and the head's shards, all rows at once."""
    rows = hidden.flatten(0, 1).detach().requires_grad_()
    weights = [w.detach().clone().requires_grad_() for w in model.head]
    logprobs, entropy = dc.linear_logprobs_and_entropy(rows, weights, tokens.flatten())
    (-(advantages.flatten() * logprobs).sum() - entropy_bonus * entropy.sum()).backward()
    return logprobs.detach().view(tokens.shape), rows.grad, [w.grad for w in weights]


def attention_step(model, tokens, layer=0, rank=0):
    """A layer's attention of one rank over whole sequences (int64 [sequences, tokens]), its inputs the embeddings: the
    keys, and the gradient of half the sum of squares of what it gives with respect to the norms' weights."""
    n, length = tokens.shape
    hq, hk, d = model.q_heads, model.kv_heads, model.dim
    y = norm(model.embedding[tokens.flatten()])
    both = torch.cat([project(part, model.qkv[layer][rank]) for part in y.split(16)]).view(n * length, hq + 2 * hk, d)
    q_norm, k_norm = (w.detach().clone().requires_grad_() for w in model.norms[layer][rank])
    positions = torch.arange(length, device=y.device, dtype=torch.int32).repeat(n)
    q, k = dc.normed_queries_and_keys(both[:, :hq], both[:, hq:hq + hk], positions, model.cos_sin, q_norm, k_norm)
    q, k, v = (t.view(n, length, -1, d).transpose(1, 2).float() for t in (q, k, both[:, hq + hk:]))
    k, v = (t.repeat_interleave(hq // hk, 1) for t in (k, v))
    score = (q @ k.transpose(2, 3) * d ** -0.5).masked_fill(torch.ones(length, length, device=y.device).triu(1).bool(), float("-inf"))
    (torch.softmax(score, -1) @ v).square().sum().mul(0.5).backward()
    return k, [q_norm.grad, k_norm.grad]


def main():
    model = NormedModel()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(0, model.vocab, (2, 32), generator=g, device="cuda")
    each, new = 6, 20
    noise = -torch.log(-torch.log(torch.rand(new, 2 * each, model.vocab, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    tokens, logprobs, hidden, _ = rollout(model, prompts, each, noise)
    same = True
    for b in range(2 * each):
        t, lp, _, _ = rollout(model, prompts[b // each:b // each + 1], 1, noise[:, b:b + 1])
        same &= torch.equal(t[:, 0], tokens[:, b]) and torch.equal(lp[:, 0], logprobs[:, b])
    print(f"2 prompts of 32 tokens, {each} samples of {new} each: alone and together the same bits: {same}")
    advantages = torch.randn(tokens.shape, generator=g, device="cuda")
    scored, rows, grads = train_step(model, tokens, hidden, advantages)
    print(f"training scores equal the rollout's: {torch.equal(scored, logprobs)}; gradient norms "
          f"{float(rows.float().norm()):.4f} (rows), {float(sum(x.float().square().sum() for x in grads)) ** 0.5:.4f} (head)")
    _, norms = attention_step(model, prompts)
    print(f"gradient norms of the norms' weights {float(norms[0].float().norm()):.4f}, {float(norms[1].float().norm()):.4f}")
    return 0 if same and torch.equal(scored, logprobs) else 1


if __name__ == "__main__":
    sys.exit(main())
