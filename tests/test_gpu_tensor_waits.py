"""Bounded waits of the tensor-core kernels: one that is made to run out (a test option lets a part of a kernel come
late) is reported by dc_check_device once, nothing of the call is left under way, and the next call is right.

All copies and products that a late call has issued complete on their own: only who waits for them gives up.
"""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reduce_copy_rank_gb300 as dc  # noqa: E402

TIMEOUT = 6
LIMIT = 2_000_000


@pytest.fixture(autouse=True)
def clean_fault_word():
    assert dc.dc_check_device() == 0, dc.last_error()
    yield
    assert dc.dc_check_device() == 0, dc.last_error()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def runs_out(call, late, what):
    with dc.options(test_tensor_late=late, wait_limit_ns=LIMIT):
        call()
        assert dc.dc_check_device() == TIMEOUT
        assert "gave up" in dc.last_error() and what in dc.last_error()
        assert "did not end" not in dc.last_error()
    assert dc.dc_check_device() == 0


def head(rows, size, widths, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(rows)
    hidden = torch.randn(rows, size, generator=g, device="cuda").to(dtype)
    weights = [(torch.randn(w, size, generator=g, device="cuda") * 2 * size ** -0.5).to(dtype) for w in widths]
    return hidden, weights, torch.randint(0, sum(widths), (rows,), generator=g, device="cuda")


@pytest.mark.parametrize("late", [1, 2, 3, 4])
@pytest.mark.parametrize("rows,size,widths", [(5, 1040, [300]), (700, 4096, [3000, 0, 2100])])
def test_log_probabilities(rows, size, widths, late):
    hidden, weights, tokens = head(rows, size, widths)
    ws = dc.linear_logprobs_workspace(rows, size, sum(widths))

    def call():
        out = [torch.full((rows,), 7.0, device="cuda") for _ in range(3)]
        dc.linear_logprobs(hidden, weights, tokens, out[0], ws, entropy=out[1], lse=out[2])
        torch.cuda.synchronize()
        return out

    want = call()
    for _ in range(2):
        runs_out(call, late, "linear head")
        assert same(call(), want)


@pytest.mark.parametrize("late", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_their_gradient(late, dtype):
    rows, size, widths = 3000, 520, [5000, 2500]
    hidden, weights, tokens = head(rows, size, widths, dtype)
    out = [torch.empty(rows, device="cuda") for _ in range(3)]
    dc.linear_logprobs(hidden, weights, tokens, out[0], dc.linear_logprobs_workspace(rows, size, 7500), entropy=out[1], lse=out[2])
    up = torch.randn(rows, device="cuda")
    ws = dc.linear_logprobs_workspace(rows, size, 7500, backward=True)

    def call():
        grads = [torch.full_like(t, 7.0) for t in (hidden, *weights)]
        dc.linear_logprobs_backward(hidden, weights, tokens, out[2], up, grads[0], grads[1:], ws, entropy=out[1], grad_entropy=up)
        torch.cuda.synchronize()
        return grads

    want = call()
    for _ in range(2):
        runs_out(call, late, "linear head")
        assert same(call(), want)


@pytest.mark.parametrize("late", [1, 2])
@pytest.mark.parametrize("page", [64, 7])  # copies by TMA, and 16 bytes each
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_to_shared_prefixes(d, page, late):
    g = torch.Generator(device="cuda").manual_seed(d + page)
    hq, hk, seqs, tokens = 76, 38, 6, 1400  # (chunks of six tiles)
    need = -(-tokens // page)
    pages = 2 * need + seqs
    kc, vc = (torch.randn(pages, page, hk, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(2 * need, generator=g, device="cuda").int().view(2, need)
    own = (2 * need + torch.arange(seqs, device="cuda")).int().view(seqs, 1)
    lengths = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([tokens, 700], [3, 0, 5, 1, 7, 2])]
    q = torch.randn(seqs, hq, d, generator=g, device="cuda").bfloat16()
    ws = dc.prefix_attention_workspace(seqs, 2, hq, hk, d, need * page, page)

    def call():
        out, lse = torch.full_like(q, 7.0), torch.full((seqs, hq), 7.0, device="cuda")
        dc.prefix_attention(q, kc, vc, table, lengths[0], own, lengths[1], out, ws, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    want = call()
    for _ in range(2):
        runs_out(call, late, "shared prefixes")
        assert same(call(), want)
