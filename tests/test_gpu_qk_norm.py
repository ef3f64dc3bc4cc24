"""Normed and rotated queries and keys, their gradient, and their way into the
paged cache, against the formulas in 64 bits.

Tolerances, from the arithmetic.  A norm's mean square is a sum of at most 512
squares in binary32 (each lane at most 32 terms in a row, then 5 pairs): within
2^-18 of itself, its root's inverse within 2^-18; a result takes three products
and a sum more and one rounding to its type (half a step, UNIT).  The gradient
subtracts mean(g w n) n, a sum like that of terms of up to n times as large: the
terms' sizes are added up beside the result.  The weights' gradient: a sum in
binary32 of as many terms as tokens and heads, a thread's in a row.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import reduce_copy_rank_gb300 as dc  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def build(n, hq, hk, d, rot, dtype="bf16", seed=0, w32=True, rows=300):
    """Heads side by side in one tensor, positions, angles, weights, upstream gradients."""
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    both = (torch.randn(n, hq + 2 * hk, d, generator=g, device="cuda") * 3).to(DT[dtype])
    pos = torch.randint(0, rows, (n,), generator=g, device="cuda").int()
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
    cs = torch.cat([angle.cos(), angle.sin()], 1).float() if rot else None
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.float32 if w32 else DT[dtype]) for _ in range(2)]
    dy = [torch.randn(n, h, d, generator=g, device="cuda").to(DT[dtype]) for h in (hq, hk)]
    return both[:, :hq], both[:, hq:hq + hk], both[:, hq + hk:], pos, cs, w, dy


def rotation(x, pos, cs, interleaved, back=False):
    if cs is None:
        return x
    rot = cs.shape[1]
    c, s = (t.double()[:, None] for t in cs[pos.long().clamp(0, len(cs) - 1)].split(rot // 2, 1))
    first = torch.arange(rot // 2, device="cuda") * (2 if interleaved else 1)
    second = first + (1 if interleaved else rot // 2)
    a, b = x[..., first], x[..., second]
    s = -s if back else s
    return x.index_copy(2, first, a * c - b * s).index_copy(2, second, b * c + a * s)


def check(have, want, size, dtype, over=2.0 ** -17):
    tol = UNIT[dtype] * want.abs() + over * size + LEAST[dtype]
    assert float(((have.double() - want).abs() - tol).max()) <= 0


def check_forward(have, x, w, pos, cs, interleaved, dtype):
    x, w = x.double(), w.double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    # (a rotated pair's terms)
    size = y.abs()
    if cs is not None:
        rot = cs.shape[1]
        first = torch.arange(rot // 2, device="cuda") * (2 if interleaved else 1)
        second = first + (1 if interleaved else rot // 2)
        pair = y[..., first].abs() + y[..., second].abs()
        size = size.index_copy(2, first, pair).index_copy(2, second, pair)
    check(have, rotation(y, pos, cs, interleaved), size, dtype)


def check_backward(dx, dw, x, w, dy, pos, cs, interleaved, dtype, keep=None):
    x, w, dy = x.double(), w.double(), dy.double()
    if keep is not None:
        dy = dy * keep[:, None, None]
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r
    g = rotation(dy, pos, cs, interleaved, back=True)
    gw = g * w
    want = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    length = dy.square().sum(-1, keepdim=True).sqrt() * w.abs().max()  # (no rotated pair is longer)
    size = r * (length + n.abs() * (gw * n).abs().mean(-1, keepdim=True) + n.abs() * length)
    check(dx, want, size, dtype)
    if dw is not None:
        terms = (dy.square().sum(-1, keepdim=True).sqrt() * n.abs()).sum((0, 1))
        kind = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[dw.dtype]
        check(dw, (g * n).sum((0, 1)), terms, kind, over=2.0 ** -16)


SHAPES = [  # tokens, query heads, key heads, dim, rotated
    (1, 1, 1, 8, 0), (1, 32, 8, 128, 128), (3, 5, 1, 64, 32), (64, 32, 8, 128, 128), (17, 12, 12, 96, 96), (33, 7, 7, 80, 32),
    (129, 3, 2, 192, 192), (40, 2, 1, 256, 64), (9, 4, 4, 512, 512), (700, 32, 8, 128, 128), (5000, 4, 1, 64, 64), (13, 3, 1, 512, 16),
    (2, 100, 3, 24, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot", SHAPES)
def test_forward_and_backward(n, hq, hk, d, rot, interleaved, dtype):
    w32 = (n + d) % 3 != 0
    q, k, _, pos, cs, w, dy = build(n, hq, hk, d, rot, dtype, w32=w32)
    out = [torch.full_like(t, 7.0, memory_format=torch.contiguous_format) for t in (q, k)]
    got = dc.qk_norm_rotate(q, k, pos, cs, *w, *out, eps=EPS, interleaved=interleaved)
    assert got[0] is out[0] and got[1] is out[1]
    for y, x, wt in zip(out, (q, k), w):
        check_forward(y, x, wt, pos, cs, interleaved, dtype)
    dx = [torch.full_like(t, 7.0) for t in dy]
    dw = [torch.full_like(t, 7.0) for t in w]
    ws = dc.qk_norm_workspace(n, hq, hk, d).fill_(255)
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dx, *dw, workspace=ws, eps=EPS, interleaved=interleaved)
    for i, x in enumerate((q, k)):
        check_backward(dx[i], dw[i], x, w[i], dy[i], pos, cs, interleaved, dtype)
    # in place, and the same bits again
    again = [t.clone() for t in (q, k)]
    dc.qk_norm_rotate(*again, pos, cs, *w, *again, eps=EPS, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(again, out))
    grads, sums = [t.clone() for t in dy], [torch.empty_like(t) for t in w]
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *grads, *grads, *sums, workspace=ws, eps=EPS, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(grads + sums, dx + dw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq,hk,d,rot,page,interleaved", [
    (64, 32, 8, 128, 128, 16, False), (1, 8, 1, 128, 128, 64, True), (130, 12, 12, 80, 32, 24, True), (7, 0, 3, 96, 96, 1, False),
    (900, 4, 2, 512, 64, 16, False), (20, 16, 4, 64, 0, 16, False)])
def test_append(n, hq, hk, d, rot, page, interleaved, dtype):
    rows = 300
    q, k, v, _, cs, w, _ = build(n, max(hq, 1), hk, d, rot, dtype, rows=rows)
    g = torch.Generator(device="cuda").manual_seed(3)
    width = -(-rows // page)
    seqs = (torch.arange(n, device="cuda") % 7).int()
    pos = (torch.arange(n, device="cuda") // 7).int()
    table = torch.randperm(7 * width, generator=g, device="cuda").int().view(7, width)
    kc, vc = (torch.randn(7 * width, page, hk, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    before = kc.clone(), vc.clone()
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format) if hq else None
    dc.kv_append(k, v, pos, seqs, table, kc, vc, q=q if hq else None, q_out=out, cos_sin=cs, interleaved=interleaved,
                 q_norm=w[0] if hq else None, k_norm=w[1], eps=EPS)
    want = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k)]
    dc.qk_norm_rotate(q, k, pos, cs, *w, *want, eps=EPS, interleaved=interleaved)
    check_forward(want[1], k, w[1], pos, cs, interleaved, dtype)
    if hq:
        assert torch.equal(out, want[0])
    where = table[seqs.long(), (pos // page).long()].long(), (pos % page).long()
    assert torch.equal(kc[where], want[1]) and torch.equal(vc[where], v)
    untouched = torch.ones(7 * width, page, dtype=torch.bool, device="cuda")
    untouched[where] = False
    assert torch.equal(kc[untouched], before[0][untouched]) and torch.equal(vc[untouched], before[1][untouched])


def test_padding_and_places_that_do_not_exist():
    q, k, v, pos, cs, w, dy = build(12, 4, 2, 64, 64, rows=200)
    pos[3], pos[5] = -1, 200
    good = [i for i in range(12) if i not in (3, 5)]
    out = [torch.full_like(t, 7.0) for t in dy]
    dc.qk_norm_rotate(q, k, pos, cs, *w, *out, eps=EPS)
    dx = [torch.full_like(t, 7.0) for t in dy]
    dw = [torch.empty_like(t) for t in w]
    ws = dc.qk_norm_workspace(12, 4, 2, 64)
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dx, *dw, workspace=ws, eps=EPS)
    for y, x, wt in zip(out, (q, k), w):
        check_forward(y[good], x[good], wt, pos[good], cs, False, "bf16")
    for t in (*out, *dx):
        assert bool((t[3] == 0).all()) and bool(torch.isnan(t[5]).all())
    assert all(bool(torch.isnan(t).all()) for t in dw)
    pos[5] = 4
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dx, *dw, workspace=ws, eps=EPS)
    keep = (pos >= 0).double()
    for i, x in enumerate((q, k)):
        check_backward(dx[i], dw[i], x, w[i], dy[i], pos, cs, False, "bf16", keep)
    # NaN in padding stays there
    q[3], dy[0][3] = math.nan, math.nan
    again, sums = [torch.empty_like(t) for t in dy], [torch.empty_like(t) for t in w]
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *again, *sums, workspace=ws, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip(again + sums, dx + dw))
    # the cache: nothing is written for padding, for a sequence or a page that does not exist
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((4, 4, 2, 64), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    at = torch.tensor([0, -1, 8, 4, 1, 2], dtype=torch.int32, device="cuda")
    seqs = torch.tensor([0, 0, 0, 1, 2, 1], dtype=torch.int32, device="cuda")
    q, k, v = q[:6], k[:6], v[:6]
    q_out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    dc.kv_append(k, v, at, seqs, table, kc, vc, q=q, q_out=q_out, cos_sin=cs, q_norm=w[0], k_norm=w[1], eps=EPS)
    assert bool((q_out[1] == 7).all()) and bool(torch.isnan(q_out[[2, 3, 4]]).all())
    check_forward(q_out[[0, 5]], q[[0, 5]], w[0], at[[0, 5]], cs, False, "bf16")
    written = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    written[0, 0] = written[2, 2] = True
    assert torch.equal(vc[0, 0], v[0]) and torch.equal(vc[2, 2], v[5])
    assert bool((kc[~written] == 5).all()) and bool((vc[~written] == 5).all())


def test_zero_heads_and_large_values():
    q, k, _, pos, cs, w, dy = build(6, 4, 2, 64, 64, "f32")
    q[0] = 0
    q[1] *= 1e15
    q[2] *= 1e-12
    out = [torch.empty_like(t) for t in dy]
    dc.qk_norm_rotate(q, k, pos, cs, *w, *out, eps=EPS)
    check_forward(out[0], q, w[0], pos, cs, False, "f32")
    assert bool((out[0][0] == 0).all())
    dx = [torch.empty_like(t) for t in dy]
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dx, eps=EPS)  # (the weights' gradients are not wanted)
    check_backward(dx[0], None, q, w[0], dy[0], pos, cs, False, "f32")


def test_rows_do_not_depend_on_the_others():
    q, k, _, pos, cs, w, dy = build(3000, 8, 2, 128, 128)
    out = [torch.empty_like(t) for t in dy]
    dx = [torch.empty_like(t) for t in dy]
    dc.qk_norm_rotate(q, k, pos, cs, *w, *out)
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dx)
    for part in (slice(0, 1), slice(2000, 2100)):
        some = [torch.empty_like(t[part]) for t in dy]
        dc.qk_norm_rotate(q[part], k[part], pos[part], cs, *w, *some)
        assert all(torch.equal(a, b[part]) for a, b in zip(some, out))
        dc.qk_norm_rotate_backward(q[part], k[part], pos[part], cs, *w, *(t[part] for t in dy), *some)
        assert all(torch.equal(a, b[part]) for a, b in zip(some, dx))


def test_no_tokens():
    q, k, v, pos, cs, w, dy = build(4, 4, 2, 64, 64)
    q, k, v, pos, dy = q[:0], k[:0], v[:0], pos[:0], [t[:0] for t in dy]
    dw = [torch.full_like(t, 7.0) for t in w]
    dc.qk_norm_rotate(q, k, pos, cs, *w, *dy)
    dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dy, *dw, workspace=dc.qk_norm_workspace(0, 4, 2, 64))
    assert all(bool((t == 0).all()) for t in dw)


@pytest.mark.parametrize("w32", [True, False])
def test_autograd(w32):
    q, k, _, pos, cs, w, dy = build(50, 4, 2, 64, 32, w32=w32)
    pos[7] = -1
    leaves = [t.clone().requires_grad_() for t in (q, k, *w)]
    out = dc.normed_queries_and_keys(leaves[0], leaves[1], pos, cs, *leaves[2:], eps=EPS, interleaved=True)
    grads = torch.autograd.grad(out, leaves, dy, retain_graph=True)
    keep = (pos >= 0).double()
    for i, x in enumerate((q, k)):
        check_backward(grads[i], grads[2 + i], x, w[i], dy[i], pos, cs, True, "bf16", keep)
    # a broadcast upstream gradient, one output alone
    (g,) = torch.autograd.grad(out[0].sum(), [leaves[0]], retain_graph=True)
    check_backward(g, None, q, w[0], torch.ones_like(dy[0]), pos, cs, True, "bf16", keep)
    # ... and one that starts off the kernels' alignment
    odd = torch.empty(dy[0].numel() + 1, device="cuda", dtype=dy[0].dtype)[1:].view_as(dy[0]).copy_(dy[0])
    (g,) = torch.autograd.grad(out[0], [leaves[0]], odd, retain_graph=True)
    assert torch.equal(g, grads[0])
    (g,) = torch.autograd.grad(out[0].sum(), [leaves[0]], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()


def test_gradient_by_differences():
    q, k, _, pos, cs, w, dy = build(10, 3, 2, 64, 64, "f32")
    leaves = [t.clone().requires_grad_() for t in (q, k, *w)]
    grads = torch.autograd.grad(dc.normed_queries_and_keys(leaves[0], leaves[1], pos, cs, *leaves[2:], eps=EPS), leaves, dy)

    def loss(q, k, wq, wk):
        s = 0.0
        for x, wt, g in ((q, wq, dy[0]), (k, wk, dy[1])):
            y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * wt
            s += float((rotation(y, pos, cs, False) * g.double()).sum())
        return s

    exact = [t.detach().double() for t in leaves]
    step = [torch.randn_like(t) * 2.0 ** -14 for t in exact]
    along = loss(*(t + s for t, s in zip(exact, step))) - loss(*(t - s for t, s in zip(exact, step)))
    have = 2 * float(sum((g.double() * s).sum() for g, s in zip(grads, step)))
    size = 2 * float(sum((g.double() * s).abs().sum() for g, s in zip(grads, step)))
    assert abs(have - along) <= 2.0 ** -16 * size  # (the third derivative's share: 2^-28)


def test_streams_graphs_and_versions():
    q, k, v, pos, cs, w, dy = build(300, 8, 2, 128, 128)
    out, dx = ([torch.empty_like(t) for t in dy] for _ in range(2))
    dw = [torch.empty_like(t) for t in w]
    ws = dc.qk_norm_workspace(300, 8, 2, 128)
    written = (*out, *dx, *dw)
    before = [t._version for t in written]

    def calls(stream=None):
        dc.qk_norm_rotate(q, k, pos, cs, *w, *out, stream=stream)
        dc.qk_norm_rotate_backward(q, k, pos, cs, *w, *dy, *dx, *dw, workspace=ws, stream=stream)

    calls()
    assert all(t._version > v for t, v in zip(written, before))
    torch.cuda.synchronize()
    want = [t.clone() for t in written]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(written, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        for t in written:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(written, want))


def test_autograd_in_a_graph():
    q, k, _, pos, cs, w, dy = build(70, 4, 2, 64, 64)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, *w)]

    def step():
        return torch.autograd.grad(dc.normed_queries_and_keys(*leaves[:2], pos, cs, *leaves[2:], eps=EPS), leaves, dy)

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
