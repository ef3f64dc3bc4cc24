"""The operators run together: samples behind shared prompts, and a training step on them."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("group_rollout", os.path.join(ROOT, "examples", "group_rollout.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def rolled(example):
    model = example.NormedModel(vocab=2051)
    g = torch.Generator(device="cuda").manual_seed(4)
    prompts = torch.randint(0, model.vocab, (2, 16), generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(12, 8, model.vocab, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    return model, prompts, noise, example.rollout(model, prompts, 4, noise)


def test_samples_do_not_depend_on_one_another(example, rolled):
    model, prompts, noise, (tokens, logprobs, hidden, _) = rolled
    assert len({tuple(t) for t in tokens.t().tolist()}) > 4  # (they do differ)
    for b in (0, 3, 6):
        t, lp, h, _ = example.rollout(model, prompts[b // 4:b // 4 + 1], 1, noise[:, b:b + 1])
        assert torch.equal(t[:, 0], tokens[:, b])
        assert torch.equal(lp[:, 0], logprobs[:, b])
        assert torch.equal(h[:, 0], hidden[:, b])


def test_training_starts_from_the_rollouts_numbers(example, rolled):
    model, _, _, (tokens, logprobs, hidden, _) = rolled
    g = torch.Generator(device="cuda").manual_seed(5)
    advantages = torch.randn(tokens.shape, generator=g, device="cuda")
    scored, rows, grads = example.train_step(model, tokens, hidden, advantages, entropy_bonus=0.02)
    assert torch.equal(scored, logprobs)
    # the same loss in 64 bits
    leaves = [t.double().detach().requires_grad_() for t in (hidden.flatten(0, 1), *model.head)]
    logp = torch.log_softmax(leaves[0] @ torch.cat(leaves[1:]).t(), 1)
    loss = -(advantages.flatten() * logp.gather(1, tokens.flatten()[:, None])[:, 0]).sum() + 0.02 * (logp.exp() * logp).sum()
    loss.backward()
    for got, want in zip((rows, *grads), (t.grad for t in leaves)):
        # two roundings to bfloat16 of independent terms: 2^-8 half steps, 0.82 of one in the mean
        assert float((got.double() - want).norm() / want.norm()) < 1.5 * 2.0 ** -8


def test_training_keys_are_the_caches(example, rolled):
    """The first layer's keys of a prompt, as a training step takes them, are bit for bit what the cache holds."""
    model, prompts, _, (_, _, _, cache) = rolled
    for rank in range(model.ranks):
        keys, grads = example.attention_step(model, prompts, rank=rank)
        group = model.q_heads // model.kv_heads
        for b in range(len(prompts)):
            held = cache.k[0][rank][cache.prefix[b].long()].flatten(0, 1)  # [tokens, heads, dim]
            assert torch.equal(keys[b, ::group].transpose(0, 1).to(torch.bfloat16), held)
        # the gradient in 64 bits, from the same projections
        n, length = prompts.shape
        hq, hk, d = model.q_heads, model.kv_heads, model.dim
        y = example.norm(model.embedding[prompts.flatten()])
        both = torch.cat([example.project(part, model.qkv[0][rank]) for part in y.split(16)]).view(n, length, -1, d).double()
        weights = [w.double().requires_grad_() for w in model.norms[0][rank]]
        c, s = (t.double()[:, None] for t in model.cos_sin[:length].split(d // 2, 1))

        def turned(x, w):
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
            a, b = x[..., :d // 2], x[..., d // 2:]
            return torch.cat([a * c - b * s, b * c + a * s], -1).transpose(1, 2)

        q, k, v = turned(both[:, :, :hq], weights[0]), turned(both[:, :, hq:hq + hk], weights[1]), both[:, :, hq + hk:].transpose(1, 2)
        k, v = (t.repeat_interleave(group, 1) for t in (k, v))
        score = (q @ k.transpose(2, 3) * d ** -0.5).masked_fill(torch.ones(length, length, device=q.device).triu(1).bool(), -torch.inf)
        (torch.softmax(score, -1) @ v).square().sum().mul(0.5).backward()
        for got, want in zip(grads, (w.grad for w in weights)):
            # queries, keys and their gradients rounded to bfloat16, 2^-8 a few times over
            assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -5
