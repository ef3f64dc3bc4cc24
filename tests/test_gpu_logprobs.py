"""token_logprobs and its gradient against the formulas in 64 bits.

Tolerances, from the arithmetic: a logit's exponent is one rounded product
and sum in binary32 and one base-2 exponential (2 ulp), at most 64 terms are
added in sequence and the rest in trees, so a row's sums are good to 2^-18 of
themselves and its logarithms to 2^-18 of (1 + log vocab); values near |z| are
rounded a few times to 2^-24 |z|.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import reduce_copy_rank_gb300 as dc  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # one rounding, relative
REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def logits(rows, vocab, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + rows * 31 + vocab)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * spread
    hot = torch.randint(0, vocab, (rows, 2), generator=g, device="cuda")
    x.scatter_add_(1, hot, torch.rand(rows, 2, generator=g, device="cuda") * 10)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tokens[::2] = hot[::2, 0]
    return x.to(dtype), tokens


def split(x, widths):
    return [s.contiguous() for s in torch.split(x, widths, dim=1)]


def uneven(vocab, P):
    cuts = sorted({0, vocab, *[(vocab * (2 * r + 1)) // (2 * P + 1) for r in range(1, P)]})
    return [b - a for a, b in zip(cuts, cuts[1:])]


def score(shards, tokens, top=0, vocab=None, temperature=1.0, index=torch.int64, stream=None):
    n = shards[0].shape[0]
    out = {k: torch.full((n,), 7.0, device="cuda") for k in ("logprobs", "entropy", "lse")}
    if top:
        out["top_logprobs"] = torch.full((n, top), 7.0, device="cuda")
        out["top_tokens"] = torch.full((n, top), -7, device="cuda", dtype=index)
    r = dc.token_logprobs(shards, tokens, vocab=vocab, temperature=temperature, stream=stream, **out)
    assert r is out["logprobs"]
    torch.cuda.synchronize()
    return out


def exact(x, tokens, temperature=1.0):
    """The scores in 64 bits, on the host."""
    z = x.cpu().to(torch.float64) * float(np.float32(1.0 / temperature))
    lse = torch.logsumexp(z, 1)
    p = (z - lse[:, None]).exp()
    ent = lse - torch.where(p > 0, p * z, 0.0).sum(1)
    return z.gather(1, tokens.cpu().long()[:, None])[:, 0] - lse, ent, lse


def check(out, x, tokens, temperature=1.0, top=0):
    lp, ent, lse = exact(x, tokens, temperature)
    z_max = float(torch.where(torch.isfinite(x) & (x > -1e4), x, 0).abs().max()) / temperature
    tol = REL * (1 + math.log(x.shape[1])) + 2.0 ** -21 * z_max
    for name, want in (("logprobs", lp), ("entropy", ent), ("lse", lse)):
        got = out[name].cpu().double()
        fine = torch.isfinite(want)
        assert torch.equal(got[~fine].nan_to_num(nan=5e30), want[~fine].nan_to_num(nan=5e30)), name
        err = (got - want)[fine].abs()
        assert err.numel() == 0 or float(err.max()) <= tol, (name, float(err.max()), tol)
    if top:
        xs = x.cpu().float()
        order = torch.from_numpy(np.argsort(-xs.numpy().astype(np.float64), axis=1, kind="stable")[:, :top].copy())
        assert torch.equal(out["top_tokens"].cpu().long(), order)
        want = torch.log_softmax(x.cpu().double() * float(np.float32(1.0 / temperature)), 1).gather(1, order)
        got = out["top_logprobs"].cpu().double()
        fine = torch.isfinite(want)
        assert torch.equal(got[~fine], want[~fine])
        assert float((got - want)[fine].abs().max()) <= tol


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,P,top", [
    (1, 1, 1, 1), (3, 2, 2, 2), (2, 31, 1, 5), (5, 2047, 1, 3), (4, 2048, 2, 8), (7, 2049, 3, 32),
    (1, 50021, 8, 20), (33, 16385, 5, 1), (340, 5003, 1, 4), (700, 3000, 2, 0), (50, 1500, 1, 32), (21, 9000, 3, 32), (2, 67187, 1, 32), (3, 20000, 2, 31), (9, 1031, 2, 20)])
def test_scores(dtype, rows, vocab, P, top):
    x, tokens = logits(rows, vocab, DT[dtype])
    out = score(split(x, uneven(vocab, P)), tokens, top=top)
    check(out, x, tokens, top=top)


@pytest.mark.parametrize("temperature", [0.5, 0.7, 1.9])
def test_temperature(temperature):
    x, tokens = logits(9, 20011, torch.bfloat16)
    check(score([x], tokens, top=6, temperature=temperature), x, tokens, temperature, top=6)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_index_types(index):
    x, tokens = logits(6, 4100, torch.float16)
    check(score([x], tokens.to(index), top=3, index=index), x, tokens, top=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bits_do_not_depend_on_batch_shards_or_layout(dtype):
    rows, vocab = 700, 33333
    x, tokens = logits(rows, vocab, DT[dtype])
    whole = score([x], tokens, top=7)
    forms = {
        "again": [x], "shards": split(x, uneven(vocab, 8)), "even shards": list(torch.split(x, 4096 + 1, dim=1)),
        "columns of a wider tensor": [torch.cat([x[:, :1], x, x[:, :3]], 1)[:, 1:vocab + 1]],
    }
    for name, shards in forms.items():
        out = score(shards, tokens, top=7)
        for k in whole:
            assert torch.equal(out[k], whole[k]), (name, k)
    for n in (1, 2, 17, 160, 400):
        out = score([x[100:100 + n]], tokens[100:100 + n], top=7)
        for k in whole:
            assert torch.equal(out[k], whole[k][100:100 + n]), (n, k)
    # neither do they depend on the alternatives asked for
    out = score([x], tokens, top=0)
    for k in ("logprobs", "entropy", "lse"):
        assert torch.equal(out[k], whole[k])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (3, 5), (7, 9), (8, 8)])
def test_every_alignment(dtype, offset, pad):
    rows, vocab = 6, 6151
    x, tokens = logits(rows, vocab, DT[dtype], seed=offset)
    store = torch.full((offset + rows * (vocab + pad) + 64,), float("nan"), device="cuda", dtype=DT[dtype])
    view = store[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    view.copy_(x)
    check(score([view], tokens, top=4), x, tokens, top=4)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("widths", [
    [1, 3, 7, 9, 2047, 2, 2031],          # several ends in one 16-byte vector, and on both sides of it
    [8, 2040, 8, 2048, 16, 1],            # ends on vectors and on segments of 2048
    [1024, 1023, 1, 5, 4, 3, 2, 1],       # three and more shards in a segment of 1024
    [2049, 4095, 6, 13],
])
@pytest.mark.parametrize("skew", [0, 1, 5])
def test_segments_of_many_shards(dtype, widths, skew):
    """Shards whose ends lie anywhere: the bits of the undivided row, and nothing beside a shard's rows."""
    vocab = sum(widths)
    x, tokens = logits(9, vocab, DT[dtype], seed=3)
    shards = []
    for r, part in enumerate(torch.split(x, widths, dim=1)):
        w, at = part.shape[1], 8 + skew * (r + 1) % 8
        room = torch.full((9, (at + w + 15) // 8 * 8 + (skew if r % 2 else 0)), float("nan"), device="cuda", dtype=DT[dtype])
        room[:, at:at + w] = part
        shards.append(room[:, at:at + w])
    got, want = score(shards, tokens, 20), score([x], tokens, 20)
    check(got, x, tokens, top=20)
    for name in want:
        assert torch.equal(got[name].view(torch.int32) if got[name].is_floating_point() else got[name],
                           want[name].view(torch.int32) if want[name].is_floating_point() else want[name]), name


def test_padding_columns_are_not_read():
    x, tokens = logits(5, 5000, torch.bfloat16)
    padded = torch.full((5, 5120), float("nan"), device="cuda", dtype=torch.bfloat16)
    padded[:, :5000] = x
    shards = split(padded, [2048, 2048, 512, 512])  # the last two partly and wholly padding
    check(score(shards, tokens, top=5, vocab=5000), x, tokens, top=5)
    empty = torch.empty(5, 0, device="cuda", dtype=torch.bfloat16)
    check(score([empty, x, empty], tokens, top=5), x, tokens, top=5)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_masked_logits(dtype):
    x, tokens = logits(8, 4500, DT[dtype])
    low = torch.finfo(DT[dtype]).min
    x[0, :2048] = -math.inf           # a whole segment
    x[1, 100:] = -math.inf
    x[2, :] = -math.inf               # nothing left
    x[3, 5:] = low                    # masks of the type's lowest value
    x[4, :] = low                     # ... everywhere: uniform
    x[5, 1:] = -math.inf              # one entry
    x[6, tokens[6]] = -math.inf       # the token itself
    tokens[1], tokens[2], tokens[3], tokens[5] = 7, 11, 2, 0
    out = score([x], tokens, top=4)
    rows = [0, 1, 3, 5, 6, 7]
    check({k: v[rows] for k, v in out.items()}, x[rows], tokens[rows], top=4)
    assert out["lse"][2] == -math.inf and out["entropy"][2] == 0 and out["logprobs"][2] == -math.inf
    assert out["top_tokens"][2].tolist() == [0, 1, 2, 3] and bool((out["top_logprobs"][2] == -math.inf).all())
    assert abs(float(out["entropy"][4]) - math.log(4500)) < 1e-4
    assert abs(float(out["logprobs"][4]) + math.log(4500)) < 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_nan_and_infinity(dtype):
    x, tokens = logits(4, 5000, DT[dtype])
    x[0, 4321] = math.nan
    x[1, 17] = math.inf
    x[2, :] = math.nan
    out = score([x], tokens, top=3)
    for k in ("logprobs", "entropy", "lse"):
        assert bool(torch.isnan(out[k][0])) and bool(torch.isnan(out[k][2])), k
    assert bool(torch.isnan(out["entropy"][1]))
    assert 4321 not in out["top_tokens"][0].tolist()
    assert int(out["top_tokens"][1, 0]) == 17
    assert out["top_tokens"][2].tolist() == [-1, -1, -1]
    check({k: v[3:] for k, v in out.items()}, x[3:], tokens[3:], top=3)


@pytest.mark.parametrize("case", ["equal", "rising", "falling", "zeros", "few values"])
def test_ties_and_sorted_rows(case):
    n = 9001
    x = {"equal": torch.full((2, n), 1.5), "rising": torch.arange(n).float().expand(2, n) / 64,
         "falling": -torch.arange(n).float().expand(2, n) / 64,
         "zeros": torch.tensor([0.0, -0.0] * n)[:n].expand(2, n),
         "few values": (torch.arange(n) * 7919 % 5).float().expand(2, n)}[case].cuda().contiguous()
    tokens = torch.tensor([0, n - 1], device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        for top in (1, 8, 32):
            check(score([x.to(dtype)], tokens, top=top), x.to(dtype), tokens, top=top)


def test_tokens_that_are_not_scored():
    x, tokens = logits(4, 3001, torch.float32)
    tokens[0], tokens[1] = -100, 3001
    out = score([x], tokens)
    assert out["logprobs"][0] == 0 and bool(torch.isnan(out["logprobs"][1]))
    ok, ent, lse = exact(x, tokens.clamp(0, 3000))
    assert torch.allclose(out["lse"].cpu().double(), lse, atol=1e-4)
    assert torch.allclose(out["entropy"].cpu().double(), ent, atol=1e-4)


def test_offsets_past_32_bits():
    stride = (1 << 31) + 8 + 1  # elements
    store = torch.empty(stride + 4096, device="cuda", dtype=torch.bfloat16)
    x, tokens = logits(2, 4000, torch.bfloat16)
    view = store.as_strided((2, 4000), (stride, 1))
    view.copy_(x)
    check(score([view], tokens, top=3), x, tokens, top=3)
    out = score([x], tokens)
    dc.token_logprobs_backward([view], tokens, out["lse"], torch.ones(2, device="cuda"), [view])
    want = [torch.empty_like(x)]
    dc.token_logprobs_backward([x], tokens, out["lse"], torch.ones(2, device="cuda"), want)
    assert torch.equal(view, want[0])


# ------------------------------------------------------------- the gradient
def exact_grad(x, tokens, g, h, temperature):
    inv = float(np.float32(1.0 / temperature))
    z = x.cpu().to(torch.float64) * inv
    lse = torch.logsumexp(z, 1, keepdim=True)
    logp = z - lse
    p = logp.exp()
    ent = -torch.where(p > 0, p * logp, 0.0).sum(1, keepdim=True)
    hot = torch.zeros_like(p)
    t = tokens.cpu().long()
    kept = t >= 0
    hot[torch.arange(len(t))[kept], t[kept]] = 1
    g = (g.cpu().double() * kept)[:, None]
    h = h.cpu().double()[:, None]
    spread = torch.where(p > 0, p * (logp + ent), 0.0)
    size = g.abs() * (hot + p) + h.abs() * torch.where(p > 0, p * (1 + logp.abs() + ent), 0.0)
    return inv * (g * (hot - p) - h * spread), inv * size


def grad_tolerance(dtype, want, size, x, temperature):
    """One rounding of the result; the statistics' absolute error (2^-18 of their size and 2^-21 |z|) times the terms
    that it enters, h p (log p + H) with both log p and H off; the type's smallest step."""
    z = float(torch.where(torch.isfinite(x), x, 0).abs().max()) / temperature
    return UNIT[dtype] * want.abs() + (2 * REL * (1 + math.log(x.shape[1])) + 2.0 ** -20 * z) * size + \
        (2.0 ** -25 if dtype == "f16" else 2.0 ** -126)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,P,temperature", [
    (1, 1, 1, 1.0), (3, 5, 2, 1.0), (2, 4099, 3, 0.7), (5, 8192, 4, 1.0), (9, 8193, 1, 1.3), (3, 40013, 8, 1.0),
    (300, 1003, 1, 1.0)])
def test_gradient(dtype, rows, vocab, P, temperature):
    x, tokens = logits(rows, vocab, DT[dtype])
    if rows > 2:
        tokens[1] = -1
    shards = split(x, uneven(vocab, P))
    out = score(shards, tokens, temperature=temperature)
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = torch.randn(rows, generator=gen, device="cuda")
    h = torch.randn(rows, generator=gen, device="cuda")
    grads = [torch.full_like(s, 7.0) for s in shards]
    r = dc.token_logprobs_backward(shards, tokens, out["lse"], g, grads, entropy=out["entropy"], grad_entropy=h,
                                   temperature=temperature)
    assert r is grads
    want, size = exact_grad(x, tokens, g, h, temperature)
    got = torch.cat(grads, 1).cpu().double()
    over = (got - want).abs() - grad_tolerance(dtype, want, size, x, temperature)
    assert float(over.max()) <= 0, float(over.max())
    # either upstream gradient alone
    only = [torch.empty_like(s) for s in shards]
    dc.token_logprobs_backward(shards, tokens, out["lse"], g, only, temperature=temperature)
    want_g, size_g = exact_grad(x, tokens, g, torch.zeros_like(h), temperature)
    over = (torch.cat(only, 1).cpu().double() - want_g).abs() - grad_tolerance(dtype, want_g, size_g, x, temperature)
    assert float(over.max()) <= 0
    dc.token_logprobs_backward(shards, tokens, out["lse"], None, only, entropy=out["entropy"], grad_entropy=h,
                               temperature=temperature)
    want_h, size_h = exact_grad(x, tokens, torch.zeros_like(g), h, temperature)
    over = (torch.cat(only, 1).cpu().double() - want_h).abs() - grad_tolerance(dtype, want_h, size_h, x, temperature)
    assert float(over.max()) <= 0
    # in place
    dc.token_logprobs_backward(shards, tokens, out["lse"], g, shards, entropy=out["entropy"], grad_entropy=h,
                               temperature=temperature)
    assert all(torch.equal(a, b) for a, b in zip(shards, grads))


def test_gradient_against_differences():
    """The directional derivative of the 64-bit scores, by central differences."""
    x, tokens = logits(3, 700, torch.float32, spread=1.0)
    out = score([x], tokens, temperature=0.8)
    g = torch.tensor([1.0, -0.5, 0.25], device="cuda")
    h = torch.tensor([0.3, 1.0, -2.0], device="cuda")
    grads = [torch.empty_like(x)]
    dc.token_logprobs_backward([x], tokens, out["lse"], g, grads, entropy=out["entropy"], grad_entropy=h, temperature=0.8)
    got = grads[0].cpu().double()
    base = x.cpu().double()

    def value(v):
        z = v * float(np.float32(1 / 0.8))
        logp = torch.log_softmax(z, 1)
        lp = logp.gather(1, tokens.cpu()[:, None])[:, 0]
        return float((g.cpu().double() * lp + h.cpu().double() * -(logp.exp() * logp).sum(1)).sum())

    gen = torch.Generator().manual_seed(5)
    for _ in range(8):
        d = torch.randn(base.shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        slope = (value(base + step * d) - value(base - step * d)) / (2 * step)
        # the differences' own error is about step^2 and 1e-16 / step; the gradient's 2^-18 of its terms
        assert abs(slope - float((got * d).sum())) <= 1e-4 * (1 + abs(slope))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,out_offset", [(0, 1), (3, 0), (1, 1), (5, 2)])
def test_gradient_alignments_and_guards(dtype, offset, out_offset):
    rows, vocab, pad = 4, 3001, 6
    x, tokens = logits(rows, vocab, DT[dtype])
    tokens[2] = vocab - 1
    tokens[3] = 0
    out = score([x], tokens)
    g = torch.ones(rows, device="cuda")
    want = [torch.empty_like(x)]
    dc.token_logprobs_backward([x], tokens, out["lse"], g, want)

    def place(o):
        store = torch.full((o + rows * (vocab + pad),), 5.0, device="cuda", dtype=DT[dtype])
        return store, store[o:].view(rows, vocab + pad)[:, :vocab]

    _, a = place(offset)
    a.copy_(x)
    store, b = place(out_offset)
    dc.token_logprobs_backward([a], tokens, out["lse"], g, [b])
    assert torch.equal(b, want[0])
    assert bool((store[:out_offset] == 5).all())
    assert bool((store[out_offset:].view(rows, -1)[:, vocab:] == 5).all())


def test_gradient_of_masked_padded_and_empty_rows():
    x, tokens = logits(5, 3000, torch.bfloat16)
    x[0, 1000:] = -math.inf
    x[1, :] = -math.inf
    x[2, 10:] = torch.finfo(torch.bfloat16).min
    x[3, 7] = math.nan
    tokens[0], tokens[1], tokens[2] = 5, 9, 3
    padded = torch.full((5, 3080), math.nan, device="cuda", dtype=torch.bfloat16)
    padded[:, :3000] = x
    shards = split(padded, [1500, 1500, 80])
    out = score(shards, tokens, vocab=3000)
    g, h = torch.ones(5, device="cuda"), torch.full((5,), 0.5, device="cuda")
    grads = [torch.full_like(s, 7.0) for s in shards]
    dc.token_logprobs_backward(shards, tokens, out["lse"], g, grads, entropy=out["entropy"], grad_entropy=h, vocab=3000)
    got = torch.cat(grads, 1)
    assert bool((got[:, 3000:] == 0).all())
    assert bool((got[1] == 0).all())
    assert bool((got[0, 1000:3000] == 0).all()) and bool((got[2, 10:3000] == 0).all())
    assert bool(torch.isnan(got[3, :3000]).all())
    rows = [0, 2, 4]
    want, size = exact_grad(x[rows], tokens[rows], g[rows], h[rows], 1.0)
    finite = x[rows].clamp(min=-100)
    over = (got[rows, :3000].cpu().double() - want).abs() - grad_tolerance("bf16", want, size, finite, 1.0)
    assert float(over.max()) <= 0


def test_gradient_shards_of_one_tensor():
    """Shards and gradients as column ranges of one tensor each: their spans meet, their elements do not."""
    x, tokens = logits(6, 4096, torch.bfloat16)
    out = score([x], tokens)
    g = torch.ones(6, device="cuda")
    want = [torch.empty_like(x)]
    dc.token_logprobs_backward([x], tokens, out["lse"], g, want)
    to = torch.empty_like(x)
    dc.token_logprobs_backward(list(x.split(1000, 1)), tokens, out["lse"], g, list(to.split(1000, 1)))
    assert torch.equal(to, want[0])
    with pytest.raises(dc.DCError, match="OVERLAP"):
        dc.token_logprobs_backward([x[:, :2000], x[:, 2000:]], tokens, out["lse"], g, [to[:, :2000], to[:, 1999:-1]])


def test_autograd():
    x, tokens = logits(7, 5001, torch.float32)
    a, b = x[:, :2000].clone().requires_grad_(), x[:, 2000:].clone().requires_grad_()
    lp, ent = dc.logprobs_and_entropy([a, b], tokens, temperature=0.9)
    (lp.sum() - 0.1 * ent.mean()).backward()  # upstream gradients that are broadcast
    y = x.double().clone().requires_grad_()
    logp = torch.log_softmax(y * float(np.float32(1 / 0.9)), 1)
    (logp.gather(1, tokens[:, None]).sum() + 0.1 * (logp.exp() * logp).sum(1).mean()).backward()
    got = torch.cat([a.grad, b.grad], 1).double()
    assert float((got - y.grad).abs().max()) <= 1e-4
    a.grad = None
    lp, _ = dc.logprobs_and_entropy([a, b], tokens)  # one of the outputs unused, one shard frozen
    lp[0].backward()
    assert bool((a.grad[1:] == 0).all()) and bool((a.grad[0] != 0).any())


def test_streams_and_graphs():
    x, tokens = logits(16, 9000, torch.bfloat16)
    want = score([x], tokens, top=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = score([x], tokens, top=2, stream=side)
    assert torch.equal(out["top_logprobs"], want["top_logprobs"])
    lp = torch.empty(16, device="cuda")
    lse = torch.empty(16, device="cuda")
    grads = [torch.empty_like(x)]
    g = torch.ones(16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dc.token_logprobs([x], tokens, lp, lse=lse)
        dc.token_logprobs_backward([x], tokens, lse, g, grads)
    y, tokens2 = logits(16, 9000, torch.bfloat16, seed=9)
    x.copy_(y)
    tokens.copy_(tokens2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lp, score([y], tokens2)["logprobs"])


def test_refusals():
    x, tokens = logits(4, 100, torch.float32)
    lp = torch.empty(4, device="cuda")
    bad = [
        (ValueError, lambda: dc.token_logprobs([], tokens, lp)),
        (ValueError, lambda: dc.token_logprobs([x.cpu()], tokens, lp)),
        (ValueError, lambda: dc.token_logprobs([x.double()], tokens, lp)),
        (ValueError, lambda: dc.token_logprobs([x.t()], tokens, lp)),
        (ValueError, lambda: dc.token_logprobs([x, x.half()], tokens, lp)),
        (ValueError, lambda: dc.token_logprobs([x, x[:3]], tokens, lp)),
        (ValueError, lambda: dc.token_logprobs([x], tokens[:3], lp)),
        (ValueError, lambda: dc.token_logprobs([x], tokens.float(), lp)),
        (ValueError, lambda: dc.token_logprobs([x], tokens, lp.half())),
        (ValueError, lambda: dc.token_logprobs([x], tokens, lp, top_tokens=torch.empty(4, 2, device="cuda"))),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, lp, vocab=101)),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, lp, vocab=0)),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, lp, temperature=0.0)),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, lp, temperature=math.nan)),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, lp, lse=lp)),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, lp, top_logprobs=torch.empty(4, 33, device="cuda"))),
        (dc.DCError, lambda: dc.token_logprobs([x], tokens, x.view(-1)[:4])),
        (ValueError, lambda: dc.token_logprobs_backward([x], tokens, lp, lp.clone(), [x, x])),
        (ValueError, lambda: dc.token_logprobs_backward([x], tokens, lp, lp.clone(), [x[:, :50]])),
        (ValueError, lambda: dc.token_logprobs_backward([x], tokens, lp, None, [x.clone()], grad_entropy=lp)),
        (dc.DCError, lambda: dc.token_logprobs_backward([x], tokens, lp, None, [x.clone()])),
        (dc.DCError, lambda: dc.token_logprobs_backward([x[:, :50]], tokens, lp, lp.clone(), [x[:, 1:51]])),
    ]
    before = dc.launch_count()
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was not refused")
    assert dc.launch_count() == before
    empty = torch.empty(0, 100, device="cuda")
    dc.token_logprobs([empty], tokens[:0], lp[:0])  # no rows: nothing to do
    assert dc.launch_count() == before


@pytest.mark.parametrize("dtype,vocab", [("f32", 4 << 20), ("bf16", (4 << 20) - 3)])
def test_largest_vocabulary(dtype, vocab):
    x, tokens = logits(2, vocab, DT[dtype])
    check(score([x], tokens, top=32), x, tokens, top=32)
    with pytest.raises(dc.DCError):
        score([torch.empty(1, (4 << 20) + 1, device="cuda", dtype=DT[dtype])], tokens[:1])


def test_second_derivative_is_refused():
    """A penalty on the gradient raises instead of counting for nothing."""
    x, tokens = logits(4, 900, torch.float32)
    x.requires_grad_()
    lp, _ = dc.logprobs_and_entropy([x], tokens)
    g, = torch.autograd.grad(lp.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        (g.square().sum() + x.square().sum()).backward()
    up = torch.ones(4, device="cuda", requires_grad=True)  # nor with respect to the upstream gradient
    lp, _ = dc.logprobs_and_entropy([x], tokens)
    g2, = torch.autograd.grad(lp, x, up, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        torch.autograd.grad(g2.sum(), up)
    lp, _ = dc.logprobs_and_entropy([x], tokens)  # the first derivative is what it was
    again, = torch.autograd.grad(lp.sum(), x)
    assert torch.equal(again, g)


@pytest.mark.parametrize("dtype,size,temperature", [
    ("bf16", 1e38, 1e-3), ("bf16", 1e38, 1.0), ("bf16", 3.0, 1e-38), ("f16", 6e4, 5e-39), ("f16", 3e3, 5e-39), ("f16", 3.0, 1e-20),
    ("f32", 1e38, 1e-3), ("f32", 3.0, 4.3e-39)])
def test_temperatures_at_which_only_the_largest_logits_count(dtype, size, temperature):
    """One step of the type is far more than the temperature: the row's largest
    logits share the probability evenly, and nothing overflows to NaN."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = ((torch.rand(5, 4100, generator=g, device="cuda") - 0.3) * size).to(DT[dtype])
    x[0] = -x[0].abs()
    x[1, :4000] = -math.inf
    x[2, ::7] = torch.finfo(DT[dtype]).min
    m = x.max(1, keepdim=True).values
    tokens = x.argmax(1)
    tokens[3] = x[3].argmin()
    out = score([x], tokens, top=2, temperature=temperature)
    ties = (x == m).sum(1).double().log().cpu()
    lp = out["logprobs"].cpu().double()
    tol = REL * (1 + math.log(4100))
    assert bool(((out["entropy"].cpu().double() - ties).abs() <= tol).all())
    rest = [0, 1, 2, 4]
    assert bool(((lp + ties)[rest].abs() <= tol).all())
    assert float(lp[3]) < -1e3
    assert not bool(torch.isnan(out["lse"]).any())
    first = torch.where(x == m, torch.arange(4100, device="cuda"), 4100).min(1).values
    assert torch.equal(out["top_tokens"][:, 0], first)


@pytest.mark.parametrize("temperature", [0.5, 1.0])
@pytest.mark.parametrize("dtype,value", [("bf16", None), ("f16", None), ("f32", None), ("f32", -2e30), ("f16", -math.inf)])
def test_gradient_of_rows_of_one_mask(dtype, value, temperature):
    """Rows of nothing but the type's lowest value (or a number like it): no
    gradient where lse is -1e30 or less, the uniform one where it is not."""
    vocab = 5000
    x = torch.full((3, vocab), torch.finfo(DT[dtype]).min if value is None else value, device="cuda", dtype=DT[dtype])
    tokens = torch.tensor([3, 4999, -1], device="cuda")
    out = score([x], tokens, temperature=temperature)
    g, h = torch.tensor([1.0, -2.0, 1.0], device="cuda"), torch.tensor([0.0, 0.5, 0.5], device="cuda")
    grads = [torch.full_like(x, 7.0)]
    dc.token_logprobs_backward([x], tokens, out["lse"], g, grads, entropy=out["entropy"], grad_entropy=h,
                               temperature=temperature)
    if float(out["lse"].max()) <= -1e30:
        assert value is not None or dtype != "f16"
        assert bool((grads[0] == 0).all())
        return
    assert dtype == "f16"
    z = torch.zeros_like(x)  # the same probabilities
    want, size = exact_grad(z, tokens, g, h, temperature)
    # lse of magnitude 65504 / temperature is off by half its last place, log p + H by that and H's own error
    lse_off = 2.0 ** -24 * 65536 / temperature + 2 * REL * (1 + math.log(vocab))
    over = (grads[0].cpu().double() - want).abs() - (UNIT[dtype] * want.abs() + lse_off * (1 + lse_off) * size + 2.0 ** -25)
    assert float(over.max()) <= 0


def test_writes_count_as_changes_in_place():
    """Autograd notices that numbers which it had kept are overwritten; a refused call changes nothing."""
    x, tokens = logits(4, 700, torch.float32)
    out = score([x], tokens)
    one = torch.ones(4, device="cuda")
    x.requires_grad_()
    p = torch.softmax(x, 1)  # (keeps its result for its gradient)
    dc.token_logprobs_backward([p], tokens, out["lse"], one, [p])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        p.sum().backward()
    y = x.detach().clone()
    outs = {"logprobs": torch.empty(4, device="cuda"), "entropy": torch.empty(4, device="cuda"),
            "lse": torch.empty(4, device="cuda"), "top_logprobs": torch.empty(4, 2, device="cuda"),
            "top_tokens": torch.empty(4, 2, device="cuda", dtype=torch.int64)}
    dc.token_logprobs([y], tokens, **outs)
    assert [t._version for t in outs.values()] == [1] * 5 and y._version == 0
    grads = [torch.empty_like(y[:, :300]), torch.empty_like(y[:, 300:])]
    with pytest.raises(dc.DCError):
        dc.token_logprobs_backward([y[:, :300], y[:, 300:]], tokens, outs["lse"], None, grads)
    assert [t._version for t in grads] == [0, 0]
    dc.token_logprobs_backward([y[:, :300], y[:, 300:]], tokens, outs["lse"], one, grads)
    assert [t._version for t in grads] == [1, 1] and y._version == 0
    with torch.inference_mode():
        z = y.clone()
        dc.token_logprobs_backward([z], tokens, outs["lse"], one, [z])
    assert torch.equal(z, torch.cat(grads, 1))


def test_autograd_of_one_output_and_of_some_shards(monkeypatch):
    """An unused output's upstream gradient is not made up, and a frozen shard stays without one."""
    from reduce_copy_rank_gb300 import operators

    seen = []
    backward = operators.token_logprobs_backward

    def spy(*a, **kw):
        seen.append((a[3] is not None, kw["grad_entropy"] is not None))
        return backward(*a, **kw)

    monkeypatch.setattr(operators, "token_logprobs_backward", spy)
    x, tokens = logits(7, 5001, torch.float32)
    up = torch.linspace(-1, 1, 7, device="cuda")
    whole = x.double().requires_grad_()
    logp = torch.log_softmax(whole, 1)
    for pick, want in (((True, False), (logp.gather(1, tokens[:, None])[:, 0] * up).sum()),
                       ((False, True), (-(logp.exp() * logp).sum(1) * up).sum())):
        exact_g, = torch.autograd.grad(want, whole, retain_graph=True)
        for frozen in (None, 0, 1):
            shards = [x[:, :2000].clone(), x[:, 2000:].clone()]
            for i, s in enumerate(shards):
                s.requires_grad_(i != frozen)
            both = dc.logprobs_and_entropy(shards, tokens)
            (both[pick.index(True)] * up).sum().backward()
            assert seen.pop() == pick and not seen
            for i, (s, w) in enumerate(zip(shards, (exact_g[:, :2000], exact_g[:, 2000:]))):
                if i == frozen:
                    assert s.grad is None
                else:
                    assert float((s.grad.double() - w).abs().max()) <= 1e-4
