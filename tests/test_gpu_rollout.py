"""The operators run together: the example's rollout and training step."""
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
    spec = importlib.util.spec_from_file_location("reproducible_rollout",
                                                  os.path.join(ROOT, "examples", "reproducible_rollout.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_rollout_does_not_depend_on_the_batch(example):
    model = example.Model(vocab=2051)
    g = torch.Generator(device="cuda").manual_seed(4)
    prompts = torch.randint(0, model.vocab, (6, 9), generator=g, device="cuda")
    tokens, logprobs, hidden = example.rollout(model, prompts, 20)
    for b in (0, 3, 5):
        t, lp, h = example.rollout(model, prompts[b:b + 1], 20)
        assert torch.equal(t[:, 0], tokens[:, b])
        assert torch.equal(lp[:, 0], logprobs[:, b])
        assert torch.equal(h[:, 0], hidden[:, b])


def test_training_starts_from_the_rollouts_numbers(example):
    model = example.Model(vocab=2051, ranks=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    prompts = torch.randint(0, model.vocab, (4, 7), generator=g, device="cuda")
    tokens, logprobs, hidden = example.rollout(model, prompts, 10)
    advantages = torch.randn(tokens.shape, generator=g, device="cuda")
    scored, grads = example.train_step(model, tokens, hidden, advantages, entropy_bonus=0.02)
    assert torch.equal(scored, logprobs)
    # the same loss in 64 bits
    weights = [w.double().detach().requires_grad_() for w in model.head]
    loss = 0.0
    for t, h, a in zip(tokens, hidden, advantages):
        logits = torch.cat([h.double() @ w.t() for w in weights], 1)
        logp = torch.log_softmax(logits, 1)
        loss = loss - (a * logp.gather(1, t[:, None])[:, 0]).sum() + 0.02 * (logp.exp() * logp).sum()
    loss.backward()
    for got, want in zip(grads, (w.grad for w in weights)):
        # logits and their gradients in bfloat16, sums of 40 rows: 2^-8 a few times over
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -5
