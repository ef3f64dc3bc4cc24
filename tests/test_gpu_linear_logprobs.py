"""linear_logprobs and its gradient against the formulas in 64 bits.

Tolerances, from the arithmetic.  A logit is a sum of exact products in
binary32, at most `size` terms added 16 at a time: it is within (size / 16 +
16) 2^-23 of sum |h||w| (each addition cut rather than rounded, at worst), and
log probabilities and lse within twice that and 2^-20 of themselves for the
exponentials, sums and logarithms; the entropy, sum p (z - lse), within the
same times 2 + its range.  The gradient: d carries the logits' error times
|g| + |e| (entropy + 2), one rounding to 16 bits (half a step, UNIT), and its
products' sums the same once more with that of the result.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import reduce_copy_rank_gb300 as dc  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    yield
    assert dc.dc_check_device() == 0, dc.last_error()  # no wait ran out


def build(rows, size, widths, vocab, dtype="bf16", seed=0, wide=0, tokens=torch.int64):
    """Hidden rows, shards (rows past `vocab` NaN), tokens; `wide`: rows that lie in wider ones."""
    g = torch.Generator(device="cuda").manual_seed(seed + 31)

    def matrix(n, scale):
        t = torch.full((n, size + wide), math.nan, device="cuda", dtype=DT[dtype])
        t[:, :size] = (torch.randn(n, size, generator=g, device="cuda") * scale).to(DT[dtype])
        return t[:, :size]

    hidden = matrix(rows, 1.0)
    weights = [matrix(w, 2.5 * size ** -0.5) for w in widths]
    first = 0
    for w in weights:
        if first + len(w) > vocab:
            w[max(0, vocab - first):] = math.nan
        first += len(w)
    tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(tokens)
    return hidden, weights, tok


def forward(hidden, weights, tokens, vocab=None, temperature=1.0, workspace=None, stream=None):
    n = len(hidden)
    lp, ent, lse = (torch.full((n,), 7.0, device="cuda") for _ in range(3))
    if workspace is None:
        workspace = dc.linear_logprobs_workspace(n, hidden.shape[1], sum(len(w) for w in weights))
    assert dc.linear_logprobs(hidden, weights, tokens, lp, workspace, entropy=ent, lse=lse, vocab=vocab,
                              temperature=temperature, stream=stream) is lp
    torch.cuda.synchronize()
    return lp, ent, lse


def truth(hidden, weights, vocab, temperature):
    w = torch.cat([x.double() for x in weights])[:vocab]
    inv = float(torch.tensor(1.0 / temperature, dtype=torch.float32))
    z = hidden.double() @ w.t() * inv
    size = hidden.double().abs() @ w.abs().t() * inv
    return z, size.amax(1) * (hidden.shape[1] / 16 + 16) * 2.0 ** -23, w, inv


def check_forward(got, hidden, weights, tokens, vocab, temperature=1.0):
    lp, ent, lse = (x.double() for x in got)
    z, err, _, _ = truth(hidden, weights, vocab, temperature)
    logp = torch.log_softmax(z, 1)
    want_lse = torch.logsumexp(z, 1)
    kept = (tokens >= 0) & (tokens < vocab)
    want_lp = logp.gather(1, tokens.clamp(0, vocab - 1).long()[:, None])[:, 0]
    want_ent = -(logp.exp() * logp).sum(1)
    assert float(((lse - want_lse).abs() - 2 * err - 2.0 ** -20 * (1 + want_lse.abs())).max()) <= 0
    over = (lp - want_lp).abs() - 2 * err - 2.0 ** -20 * (1 + want_lp.abs() + want_lse.abs())
    assert float(torch.where(kept, over, -1.0).max()) <= 0
    assert float(((ent - want_ent).abs() - 2 * (2 + want_ent) * err - 2.0 ** -19 * (1 + want_lse.abs() + want_ent)).max()) <= 0
    assert bool((lp[tokens < 0] == 0).all()) and bool(torch.isnan(lp[tokens >= vocab]).all())


SHAPES = [  # rows, hidden size, shards, vocabulary
    (1, 8, [1], 1), (1, 64, [2], 2), (2, 16, [255], 255), (3, 72, [256], 256), (127, 64, [257], 257), (128, 128, [300, 211], 511),
    (129, 64, [0, 5, 0, 700], 705), (300, 1000, [1000, 1, 513], 1514), (5, 512, [2050, 2049], 4099), (64, 200, [640, 640, 640], 1501),
    (40, 64, [300, 300, 300], 290), (257, 1032, [4096], 4096), (130, 64, [33000], 33000), (9, 4096, [16384, 20], 16404)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,size,widths,vocab", SHAPES)
def test_forward(rows, size, widths, vocab, dtype):
    a = build(rows, size, widths, vocab, dtype)
    check_forward(forward(*a, vocab=vocab), *a, vocab)


@pytest.mark.parametrize("temperature", [0.3, 0.7, 1.7])
def test_temperature_strides_and_narrow_tokens(temperature):
    a = build(70, 136, [500, 300], 777, wide=24, tokens=torch.int32)
    a[2][3], a[2][5], a[2][7] = -1, 777, -100
    check_forward(forward(*a, vocab=777, temperature=temperature), *a, 777, temperature)


def test_far_maxima():
    """Logits of hundreds, and a token far ahead of all others."""
    hidden, weights, tokens = build(33, 128, [900], 900)
    hidden *= 40
    weights[0][77] = hidden[5]
    check_forward(forward(hidden, weights, tokens), hidden, weights, tokens, 900)


def test_nan_and_infinity_stay_in_their_rows():
    hidden, weights, tokens = build(200, 64, [600], 600)
    want = forward(hidden, weights, tokens)
    hidden[3, 7] = math.nan
    hidden[150, 0] = math.inf
    got = forward(hidden, weights, tokens)
    for g, w in zip(got, want):
        assert bool(torch.isnan(g[[3, 150]]).all())
        keep = [i for i in range(200) if i not in (3, 150)]
        assert torch.equal(g[keep], w[keep])


def test_bits_do_not_depend_on_rows_or_shards():
    hidden, weights, tokens = build(300, 520, [2900], 2900)
    want = forward(hidden, weights, tokens)
    for part in (slice(0, 1), slice(7, 8), slice(100, 229), slice(290, 300)):
        got = forward(hidden[part], weights, tokens[part])
        assert all(torch.equal(g, w[part]) for g, w in zip(got, want))
    for cuts in ([256], [512, 1024, 2816], [0, 256, 256, 2560, 2900]):
        shards = [weights[0][a:b].clone() for a, b in zip([0] + cuts, cuts + [2900])]
        got = forward(hidden, shards, tokens)
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def upstream(n, seed=0, entropy=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    gl = torch.randn(n, generator=g, device="cuda")
    return gl, torch.randn(n, generator=g, device="cuda") * 0.2 if entropy else None


def backward(hidden, weights, tokens, vocab, gl, ge, temperature=1.0, hidden_too=True, weights_too=True, saved=None, workspace=None):
    lp, ent, lse = saved or forward(hidden, weights, tokens, vocab, temperature)
    size = hidden.shape[1]
    gh = torch.full((len(hidden), size + 8), 7.0, device="cuda", dtype=hidden.dtype)[:, :size] if hidden_too else None
    gw = [torch.full((len(w), size), 7.0, device="cuda", dtype=hidden.dtype) for w in weights] if weights_too else None
    if workspace is None:
        workspace = dc.linear_logprobs_workspace(len(hidden), size, sum(len(w) for w in weights), backward=True)
    dc.linear_logprobs_backward(hidden, weights, tokens, lse, gl, gh, gw, workspace, entropy=ent, grad_entropy=ge, vocab=vocab,
                                temperature=temperature)
    torch.cuda.synchronize()
    return gh, gw


def check_backward(got, hidden, weights, tokens, vocab, gl, ge, temperature=1.0, dtype="bf16"):
    gh, gw = got
    z, err, w, inv = truth(hidden, weights, vocab, temperature)
    logp = torch.log_softmax(z, 1)
    p = logp.exp()
    ent = -(p * logp).sum(1, keepdim=True)
    kept = tokens >= 0
    zero = torch.zeros(len(hidden), device="cuda", dtype=torch.float64)
    g = (torch.where(kept, gl.double(), 0.0) if gl is not None else zero)[:, None]
    e = (ge.double() if ge is not None else zero)[:, None]
    d = -p * (g + e * (logp + ent))
    hot = tokens.clamp(min=0).long()[:, None]
    d = d.scatter_add(1, hot, g) * inv
    # what d may be off by: the logits' and lse's errors, and one rounding to 16 bits
    loss = (3 * err[:, None] + 2.0 ** -18) * p * (g.abs() + e.abs() * (logp.abs() + ent + 2)) * inv + (UNIT[dtype] + 2.0 ** -20) * d.abs()
    if dtype == "f16":  # below 2^-14 of d's unit (largest 2^14 or more): half of 2^-24
        loss = loss + 2.0 ** -38 * (g.abs() + 16 * e.abs()).amax() * inv
    x = hidden.double()
    pairs = []
    if gh is not None:
        pairs.append((gh.double(), d @ w, loss @ w.abs(), d.abs() @ w.abs()))
    if gw is not None:
        whole = torch.cat([t.double() for t in gw])
        assert bool((whole[vocab:] == 0).all())
        pairs.append((whole[:vocab], d.t() @ x, loss.t() @ x.abs(), d.abs().t() @ x.abs()))
    for have, want, off, size in pairs:
        tol = UNIT[dtype] * (want.abs() + off) + off + 2.0 ** -15 * size + (2.0 ** -24 if dtype == "f16" else 2.0 ** -133)
        assert float(((have - want).abs() - tol).max()) <= 0
        if len(have) > 1 and have.shape[1] > 8 and dtype == "bf16":  # both roundings, as independent errors: 0.82 of half a step
            assert float((have - want).norm()) <= 1.5 * UNIT[dtype] * float(want.norm())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,size,widths,vocab", SHAPES)
def test_backward(rows, size, widths, vocab, dtype):
    a = build(rows, size, widths, vocab, dtype, seed=1)
    if rows > 8:
        a[2][::5] = -100
    up = upstream(rows)
    check_backward(backward(*a, vocab, *up), *a, vocab, *up, dtype=dtype)


@pytest.mark.parametrize("gl,ge,hidden_too,weights_too", [
    (True, False, True, True), (False, True, True, True), (True, True, True, False), (True, True, False, True)])
def test_parts_of_the_gradient(gl, ge, hidden_too, weights_too):
    a = build(70, 136, [500, 300], 777, wide=24, tokens=torch.int32)
    g, e = upstream(70)
    up = (g if gl else None, e if ge else None)
    got = backward(*a, 777, *up, temperature=0.7, hidden_too=hidden_too, weights_too=weights_too)
    assert (got[0] is None) == (not hidden_too) and (got[1] is None) == (not weights_too)
    check_backward(got, *a, 777, *up, temperature=0.7)


def test_half_precision_keeps_small_upstream_gradients():
    a = build(60, 64, [900], 900, "f16")
    g, e = upstream(60)
    for unit in (2.0 ** -20, 2.0 ** 12):
        up = (g * unit, e * unit)
        check_backward(backward(*a, 900, *up), *a, 900, *up, dtype="f16")


def test_backward_bits_do_not_depend_on_the_other_rows():
    a = build(300, 520, [17000], 17000)
    up = upstream(300)
    saved = forward(*a)
    want = backward(*a, 17000, *up, saved=saved)
    again = backward(*a, 17000, *up, saved=saved)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1][0], again[1][0])
    for part in (slice(0, 1), slice(100, 229)):
        got = backward(a[0][part], a[1], a[2][part], 17000, *(u[part] for u in up), saved=[x[part] for x in saved], weights_too=False)
        assert torch.equal(got[0], want[0][part])


def test_no_rows():
    hidden, weights, tokens = build(3, 64, [100, 50], 140)
    empty = hidden[:0], weights, tokens[:0]
    ws = dc.linear_logprobs_workspace(0, 64, 150, backward=True)
    lp = torch.empty(0, device="cuda")
    dc.linear_logprobs(*empty, lp, ws, vocab=140)
    grads = [torch.full_like(w, 3.0) for w in weights]
    dc.linear_logprobs_backward(*empty, lp, lp, torch.empty_like(empty[0]), grads, ws, vocab=140)
    assert all(bool((g == 0).all()) for g in grads)


def test_rows_without_a_finite_logit_have_no_gradient():
    hidden, weights, tokens = build(20, 64, [300], 300)
    saved = forward(hidden, weights, tokens)
    want = backward(hidden, weights, tokens, 300, *upstream(20), saved=saved)
    saved[2][[3, 11]] = -math.inf
    got = backward(hidden, weights, tokens, 300, *upstream(20), saved=saved)
    keep = [i for i in range(20) if i not in (3, 11)]
    assert bool((got[0][[3, 11]] == 0).all()) and torch.equal(got[0][keep], want[0][keep])
    assert bool(torch.isfinite(got[1][0]).all())


def test_one_workspace_for_smaller_calls_and_its_contents_do_not_matter():
    ws = dc.linear_logprobs_workspace(200, 128, 3000, backward=True).fill_(255)
    fs = dc.linear_logprobs_workspace(200, 128, 3000).fill_(255)
    for rows, widths in ((200, [1500, 1500]), (7, [33]), (130, [2999]), (200, [3000])):
        a = build(rows, 128, widths, sum(widths))
        up = upstream(rows)
        check_forward(forward(*a, workspace=fs), *a, sum(widths))
        check_backward(backward(*a, sum(widths), *up, workspace=ws), *a, sum(widths), *up)


def test_autograd_and_differences():
    hidden, weights, tokens = build(24, 64, [200, 100], 280)
    leaves = [hidden.contiguous().requires_grad_(), *(w[:min(len(w), 280 - 200 * i)].contiguous().requires_grad_() for i, w in enumerate(weights))]
    lp, ent = dc.linear_logprobs_and_entropy(leaves[0], leaves[1:], tokens, temperature=0.8)
    g, e = upstream(24)
    grads = torch.autograd.grad((lp * g + ent * e).sum(), leaves)
    check_backward((grads[0], grads[1:]), leaves[0].detach(), [w.detach() for w in leaves[1:]], tokens, 280, g, e, temperature=0.8)
    # along a direction, by differences in 64 bits of the formula
    def loss(x, w):
        logp = torch.log_softmax(x @ torch.cat(w).t() / 0.8, 1)
        return float((logp.gather(1, tokens[:, None])[:, 0] * g - (logp.exp() * logp).sum(1) * e).sum())
    exact = [t.detach().double() for t in leaves]
    step = [torch.randn_like(t) * 2.0 ** -12 for t in exact]
    up = loss(exact[0] + step[0], [w + s for w, s in zip(exact[1:], step[1:])])
    down = loss(exact[0] - step[0], [w - s for w, s in zip(exact[1:], step[1:])])
    along = float(sum((x.double() * s).sum() for x, s in zip(grads, step))) * 2
    size = float(sum((x.double() * s).square().sum() for x, s in zip(grads, step))) ** 0.5 * 2
    assert abs(along - (up - down)) <= 4 * UNIT["bf16"] * size + 2.0 ** -16 * abs(up - down)


def test_autograd_uses_what_is_asked_for():
    hidden, weights, tokens = build(10, 64, [300], 300)
    x = hidden.clone().requires_grad_()
    lp, ent = dc.linear_logprobs_and_entropy(x, weights, tokens)
    lp.sum().backward()  # (a broadcast upstream gradient, no entropy, frozen weights)
    check_backward((x.grad, None), hidden, weights, tokens, 300, torch.ones(10, device="cuda"), None)
    w = weights[0].clone().requires_grad_()
    lp, ent = dc.linear_logprobs_and_entropy(x, [w], tokens)
    (g,) = torch.autograd.grad(ent.sum(), [w], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
    lp, ent = dc.linear_logprobs_and_entropy(x, [w], tokens)
    dc.linear_logprobs(hidden, weights, tokens, torch.empty(10, device="cuda"), dc.linear_logprobs_workspace(10, 64, 300))
    w.data.mul_(1)  # (not a change that autograd sees)
    lp.sum().backward()


def test_written_tensors_count_as_changed():
    hidden, weights, tokens = build(10, 64, [300], 300)
    saved = forward(hidden, weights, tokens)
    out = [torch.empty_like(hidden), torch.empty_like(weights[0])]
    before = [t._version for t in (*saved, *out)]
    ws = dc.linear_logprobs_workspace(10, 64, 300, backward=True)
    dc.linear_logprobs(hidden, weights, tokens, saved[0], ws, entropy=saved[1], lse=saved[2])
    dc.linear_logprobs_backward(hidden, weights, tokens, saved[2], saved[0], out[0], [out[1]], ws)
    assert all(t._version > v for t, v in zip((*saved, *out), before))


def test_streams_and_graphs():
    a = build(140, 264, [700, 900], 1555)
    up = upstream(140)
    want = forward(*a, vocab=1555)
    grads = backward(*a, 1555, *up, saved=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = forward(*a, vocab=1555, stream=side)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    out = [torch.empty(140, device="cuda") for _ in range(3)]
    gh, gw = torch.empty_like(a[0]), [torch.empty_like(w) for w in a[1]]
    fs, bs = dc.linear_logprobs_workspace(140, 264, 1600), dc.linear_logprobs_workspace(140, 264, 1600, backward=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dc.linear_logprobs(a[0], a[1], a[2], out[0], fs, entropy=out[1], lse=out[2], vocab=1555)
        dc.linear_logprobs_backward(a[0], a[1], a[2], out[2], up[0], gh, gw, bs, entropy=out[1], grad_entropy=up[1], vocab=1555)
    for _ in range(3):
        for t in (*out, gh, *gw):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(out, want))
        assert torch.equal(gh, grads[0]) and all(torch.equal(g, w) for g, w in zip(gw, grads[1]))


def test_offsets_past_32_bits():
    """Weights of more than 2^32 bytes."""
    size, vocab = 8192, 300000
    w = torch.zeros(vocab, size, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(2)
    hidden = torch.randn(3, size, generator=g, device="cuda").to(torch.bfloat16)
    some = torch.tensor([0, 5, 262143, 262144, 270001, 299999], device="cuda")
    w[some] = (torch.randn(6, size, generator=g, device="cuda") * 0.03).to(torch.bfloat16)
    tokens = torch.tensor([299999, 262144, 9], device="cuda")
    a = hidden, [w], tokens
    z = hidden.double() @ w[some].double().t()
    lse = torch.logsumexp(torch.cat([z, torch.full((3, 1), math.log(vocab - 6), device="cuda", dtype=torch.float64)], 1), 1)
    saved = forward(*a)
    assert float((saved[2].double() - lse).abs().max()) < 1e-3
    assert abs(float(saved[0][0].double() - (z[0, 5] - lse[0]))) < 1e-3
    up = upstream(3, entropy=False)
    gh, gw = backward(*a, vocab, *up, saved=saved)
    p = (z - lse[:, None]).exp()
    hot = (some[None] == tokens[:, None]).double()
    d = up[0].double()[:, None] * (hot - p)
    want = d.t() @ hidden.double()
    tol = UNIT["bf16"] * want.abs() + (UNIT["bf16"] + 2.0 ** -8) * (d.abs().t() @ hidden.double().abs())
    assert bool(((gw[0][some].double() - want).abs() <= tol).all())
    want = d @ w[some].double()
    tol = UNIT["bf16"] * want.abs() + (UNIT["bf16"] + 2.0 ** -8) * (d.abs() @ w[some].double().abs())
    assert bool(((gh.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tokens_that_many_rows_share(dtype):
    a = build(700, 72, [300, 500], 790, dtype, seed=4)
    up = upstream(700)
    for tokens in (torch.full((700,), 311, device="cuda"), torch.arange(700, device="cuda") % 40 + 280):
        b = (*a[:2], tokens.to(a[2].dtype))
        check_backward(backward(*b, 790, *up), *b, 790, *up, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sums_over_many_rows(dtype):
    """More rows than one sum on the tensor cores takes."""
    rows = 60000
    a = build(rows, 72, [300, 257], 557, dtype, seed=5)
    up = upstream(rows)
    ws = dc.linear_logprobs_workspace(rows, 72, 557, backward=True).fill_(255)
    check_backward(backward(*a, 557, *up, workspace=ws), *a, 557, *up, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_tokens_gradient_is_rounded_once(dtype):
    """Where the tokens' own columns make a gradient up (flat rows: the others have 2^-12 of its square), it has the
    error of its last rounding: half a step at most, UNIT / sqrt(3) in the root mean square."""
    hidden, weights, tokens = build(200, 64, [5000], 5000, dtype, seed=6)
    weights[0].mul_(2.0 ** -6)
    g, _ = upstream(200)
    gh, (gw,) = backward(hidden, weights, tokens, 5000, g, None)
    z, _, w, _ = truth(hidden, weights, 5000, 1.0)
    d = -torch.softmax(z, 1) * g.double()[:, None]
    d.scatter_add_(1, tokens.long()[:, None], g.double()[:, None])
    for have, want in ((gh, d @ w), (gw, d.t() @ hidden.double())):
        assert float((have.double() - want).norm()) <= 0.6 * UNIT[dtype] * float(want.norm())


def test_rows_without_upstream_gradients_have_none():
    """... whatever they hold.  (The weights' gradient is a product with all hidden rows: those have to be finite.)"""
    hidden, weights, tokens = build(200, 64, [400], 400)
    masked = torch.arange(200, device="cuda") % 3 == 0
    tokens[masked] = -100
    g, e = upstream(200)
    e[masked] = 0
    saved = forward(hidden, weights, tokens)
    want = backward(hidden, weights, tokens, 400, g, e, saved=saved)
    hidden[masked] = math.nan
    saved[2][masked] = math.nan
    saved[1][masked] = 0
    got = backward(hidden, weights, tokens, 400, g, e, saved=saved, weights_too=False)
    assert torch.equal(got[0], want[0]) and bool((got[0][masked] == 0).all())


def test_autograd_in_a_graph():
    hidden, weights, tokens = build(50, 64, [300, 200], 500)
    leaves = [t.detach().clone().requires_grad_() for t in (hidden, *weights)]
    g, e = upstream(50)

    def step():
        lp, ent = dc.linear_logprobs_and_entropy(leaves[0], leaves[1:], tokens)
        return torch.autograd.grad((lp * g + ent * e).sum(), leaves)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def shared_tokens(kind, rows, vocab, g):
    if kind == "one":
        return torch.full((rows,), vocab // 3, device="cuda")
    if kind == "half":
        return torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, vocab // 3,
                           torch.randint(0, vocab, (rows,), generator=g, device="cuda"))
    if kind == "counts":  # token k belongs to k rows: 1, 2, ..., as long as there are rows
        return torch.repeat_interleave(torch.arange(200, device="cuda"), torch.arange(200, device="cuda"))[:rows][torch.randperm(rows, generator=g, device="cuda")]
    p = 1 / torch.arange(1, vocab + 1, device="cuda").double()  # as text has them
    return torch.multinomial(p, rows, replacement=True, generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,size,widths,kind", [
    (63, 264, [300], "one"), (64, 520, [300, 40], "half"), (65, 520, [300, 40], "half"), (80, 72, [300], "one"), (16, 64, [50], "one"),
    (4095, 264, [513, 700], "half"), (4500, 264, [600], "counts"), (9000, 72, [700], "one"), (9000, 520, [400, 400], "zipf"),
    (30000, 72, [26000], "zipf"), (2500, 8, [1000], "zipf")])
def test_tokens_that_any_number_of_rows_share(rows, size, widths, kind, dtype):
    """Some of the rows (half of those that share) without a gradient."""
    vocab = sum(widths)
    hidden, weights, tokens = build(rows, size, widths, vocab, dtype, seed=7)
    g = torch.Generator(device="cuda").manual_seed(rows)
    tokens = shared_tokens(kind, rows, vocab, g)
    gl, ge = upstream(rows)
    none = torch.rand(rows, generator=g, device="cuda") < 0.4
    gl[none], ge[none] = 0, 0
    a = hidden, weights, tokens
    ws = dc.linear_logprobs_workspace(rows, size, vocab, backward=True).fill_(255)
    saved = forward(*a)
    want = backward(*a, vocab, gl, ge, saved=saved, workspace=ws)
    check_backward(want, *a, vocab, gl, ge, dtype=dtype)
    again = backward(*a, vocab, gl, ge, saved=saved, workspace=ws)
    assert torch.equal(want[0], again[0]) and all(torch.equal(x, y) for x, y in zip(want[1], again[1]))


def test_the_sum_of_shared_tokens_is_rounded_once():
    """As test_the_tokens_gradient_is_rounded_once, for tokens that 9 and 900 rows share: rows that point the same way."""
    hidden, weights, _ = build(1800, 64, [5000], 5000, seed=6)
    weights[0].mul_(2.0 ** -6)
    hidden.copy_(hidden[:1] + 0.25 * hidden)
    for each in (9, 900):
        tokens = torch.arange(1800, device="cuda") // each
        gl = upstream(1800)[0].abs()
        _, (gw,) = backward(hidden, weights, tokens, 5000, gl, None)
        z, _, _, _ = truth(hidden, weights, 5000, 1.0)
        d = -torch.softmax(z, 1) * gl.double()[:, None]
        d.scatter_add_(1, tokens[:, None], gl.double()[:, None])
        want = (d.t() @ hidden.double())[:1800 // each]
        assert float((gw[:1800 // each].double() - want).norm()) <= 0.6 * UNIT["bf16"] * float(want.norm())


@pytest.mark.parametrize("upstream_too", [True, False])
def test_no_wait_runs_out_where_thousands_of_rows_share_a_token(upstream_too):
    rows, size, vocab = 12000, 1024, 20000
    hidden, weights, tokens = build(rows, size, [vocab], vocab, seed=8)
    half = torch.arange(rows, device="cuda") % 2 == 0
    tokens[half] = 7
    gl, ge = upstream(rows)
    if not upstream_too:
        gl[half], ge[half] = 0, 0
    a = hidden, weights, tokens
    saved = forward(*a)
    with dc.options(wait_limit_ns=2_000_000):
        got = backward(*a, vocab, gl, ge, saved=saved)
        assert dc.dc_check_device() == 0, dc.last_error()
    check_backward(got, *a, vocab, gl, ge)


@pytest.mark.parametrize("dtype,power,temperature", [
    ("bf16", 0, 1e-7), ("bf16", 0, 1e-9), ("bf16", 0, 1e-20), ("bf16", 0, 1e-36), ("bf16", 0, 4.3e-39), ("bf16", 27, 1.0), ("bf16", 60, 1.0),
    ("bf16", 105, 1e-3), ("f16", 12, 1e-9), ("f16", 0, 4.3e-39)])
def test_temperatures_and_logits_at_which_only_the_largest_count(dtype, power, temperature):
    """Whole numbers times a power of two, so that the logits are exact: the largest of a row share the probability
    evenly, and nothing overflows to NaN."""
    g = torch.Generator(device="cuda").manual_seed(3)
    hidden = torch.randint(-3, 4, (140, 72), generator=g, device="cuda")
    weights = [torch.randint(-3, 4, (n, 72), generator=g, device="cuda") for n in (700, 513)]
    z = hidden.double() @ torch.cat(weights).double().t()
    hidden = (hidden.double() * 2.0 ** power).to(DT[dtype])
    tokens = z.argmax(1)
    tokens[7], tokens[100] = z[7].argmin(), z[100].argmin()
    lp, ent, lse = forward(hidden, [w.to(DT[dtype]) for w in weights], tokens, temperature=temperature)
    ties = (z == z.amax(1, keepdim=True)).sum(1).double().log()
    tol = 2.0 ** -20 * (1 + math.log(1213))
    assert int((ties > 0).sum()) > 3
    assert float((ent.double() - ties).abs().max()) <= tol
    rest = [i for i in range(140) if i not in (7, 100)]
    assert float((lp.double() + ties)[rest].abs().max()) <= tol
    assert bool((lp[[7, 100]] < -1e6).all()) and not bool(torch.isnan(lse).any())


def test_rows_of_nothing_but_minus_infinity():
    hidden, weights, tokens = build(5, 64, [300], 300)
    weights[0].abs_().neg_()
    hidden[1] = 3e38  # (its logits are sums that leave binary32)
    tokens[1] = 7
    lp, ent, lse = forward(hidden, weights, tokens)
    assert float(lse[1]) == -math.inf and float(lp[1]) == -math.inf and float(ent[1]) == 0
    keep = [0, 2, 3, 4]
    check_forward([t[keep] for t in (lp, ent, lse)], hidden[keep], weights, tokens[keep], 300)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("entropy", [True, False])
def test_tokens_past_the_vocabulary_have_no_gradient_that_is_a_number(entropy, dtype):
    """... unless nothing comes from above: what token_logprobs_backward of the same logits gives their rows."""
    hidden, weights, tokens = build(90, 64, [300, 100], 380, dtype)
    gl, ge = upstream(90, entropy=entropy)
    saved = forward(hidden, weights, tokens, 380)
    tokens[[5, 40]] = torch.tensor([380, 5000], device="cuda")
    tokens[70] = 399
    gl[70] = 0
    if entropy:
        ge[70] = 0
    gh, gw = backward(hidden, weights, tokens, 380, gl, ge, saved=saved)
    bad = torch.tensor([5, 40], device="cuda")
    logits = [(hidden.double() @ w.nan_to_num().double().t()).to(DT[dtype]) for w in weights]
    grads = [torch.empty_like(x) for x in logits]
    dc.token_logprobs_backward(logits, tokens, saved[2], gl, grads, entropy=saved[1], grad_entropy=ge, vocab=380)
    assert all(bool(torch.isnan(g[bad][:, :w]).all()) for g, w in zip(grads, (300, 80)))
    assert bool(torch.isnan(gh[bad]).all()) and bool((gh[70] == 0).all())
    keep = [i for i in range(90) if i not in (5, 40)]
    assert bool(torch.isfinite(gh[keep]).all())
    assert bool(torch.isnan(gw[0]).all()) and bool((gw[1][80:] == 0).all())
    a = hidden[keep], weights, torch.where(tokens[keep] >= 380, -1, tokens[keep])
    check_backward((backward(*a, 380, gl[keep], ge[keep] if entropy else None, saved=[t[keep] for t in saved])[0], None), *a, 380,
                   gl[keep], ge[keep] if entropy else None, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_probabilities_from_a_large_lse(dtype):
    """Whole numbers and a temperature of 2^-14, so that z is exact: log p = z - lse is off by the rounding of lse that
    it is given and no more, p by 2^-20 of itself for the exponential, and d by half a step."""
    g = torch.Generator(device="cuda").manual_seed(12)
    hidden = torch.randint(-3, 4, (100, 72), generator=g, device="cuda").to(DT[dtype])
    weights = [torch.randint(-3, 4, (900, 72), generator=g, device="cuda").to(DT[dtype])]
    tokens = torch.full((100,), -1, device="cuda")
    tokens[::2] = (hidden.float() @ weights[0].float().t()).argmax(1)[::2]
    saved = forward(hidden, weights, tokens, temperature=2.0 ** -14)
    assert float(saved[2].max()) > 2e6
    up = upstream(100)[0] * 2.0 ** -8  # (gradients that binary16 holds)
    gh, (gw,) = backward(hidden, weights, tokens, 900, up, None, temperature=2.0 ** -14, saved=saved)
    z = hidden.double() @ weights[0].double().t() * 2.0 ** 14
    kept = (tokens >= 0).double()[:, None]
    d = -(z - saved[2].double()[:, None]).exp() * up.double()[:, None] * kept
    loss = d.abs() * (UNIT[dtype] + 2.0 ** -20)
    d = (d + torch.nn.functional.one_hot(tokens.clamp(min=0), 900) * up.double()[:, None] * kept) * 2.0 ** 14
    loss = loss * 2.0 ** 14 + d.abs() * UNIT[dtype]
    for have, want, off in ((gh, d @ weights[0].double(), loss @ weights[0].double().abs()), (gw, d.t() @ hidden.double(), loss.t() @ hidden.double().abs())):
        tol = UNIT[dtype] * (want.abs() + off) + off + 2.0 ** -10
        assert float(((have.double() - want).abs() - tol).max()) <= 0
