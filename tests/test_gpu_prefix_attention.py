"""prefix_attention against the formulas in 64 bits.

Tolerances, from the arithmetic.  The prefix's weights are rounded to 16 bits
(half a step, UNIT) before they meet the values, so the output is within UNIT of
sum p |v| (2^-12 of it for the scores' and exponentials' binary32), and is
rounded once more.  As the weights' errors are independent, the whole is within
1.5 UNIT in the root mean square (0.82 expected).  lse: binary32 throughout.
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


def build(prefixes, own, hq, hk, d, page, dtype="bf16", seed=0, layout="token"):
    """Prefix lengths and own lengths (in groups of equal size) as tables over one shuffled pool; slots that hold
    no token are NaN, entries past an end -1."""
    g = torch.Generator(device="cuda").manual_seed(seed + 41)
    lengths = list(prefixes) + list(own)
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").int()

    def table(rows, at):
        t = torch.full((len(rows), max(1, max(need[r] for r in rows))), -1, dtype=torch.int32, device="cuda")
        for i, r in enumerate(rows):
            t[i, :need[r]] = order[at:at + need[r]]
            at += need[r]
        return t, at

    pt, at = table(range(len(prefixes)), 0)
    ot, _ = table(range(len(prefixes), len(lengths)), at)
    if layout == "token":
        kc, vc = (torch.randn(pages, page, hk, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    elif layout == "head":  # heads outside tokens
        kc, vc = (torch.randn(pages, hk, page, d, generator=g, device="cuda").to(DT[dtype]).transpose(1, 2) for _ in range(2))
    else:  # keys and values of a page side by side in one tensor
        both = torch.randn(pages, 2, page, hk, d, generator=g, device="cuda").to(DT[dtype])
        kc, vc = both[:, 0], both[:, 1]
    held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for t, ns in ((pt, prefixes), (ot, own)):
        for i, n in enumerate(ns):
            for j in range(-(-n // page)):
                held[t[i, j].long(), :min(page, n - j * page)] = True
    kc[~held] = math.nan
    vc[~held] = math.nan
    q = torch.randn(len(own), hq, d, generator=g, device="cuda").to(DT[dtype])
    as_int = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (prefixes, own)]
    return q, kc, vc, pt, as_int[0], ot, as_int[1]


def attend(q, kc, vc, pt, pl, ot, ol, scale=None, workspace=None, stream=None):
    n, hq, d = q.shape
    page = kc.shape[1]
    if workspace is None:
        workspace = dc.prefix_attention_workspace(n, len(pt), hq, kc.shape[2], d, pt.shape[1] * page, ot.shape[1] * page)
    out = torch.full((n, hq, d), 7.0, device="cuda", dtype=q.dtype)
    lse = torch.full((n, hq), 7.0, device="cuda")
    assert dc.prefix_attention(q, kc, vc, pt, pl, ot, ol, out, workspace, scale=scale, lse=lse, stream=stream) is out
    torch.cuda.synchronize()
    return out, lse


def check(got, q, kc, vc, pt, pl, ot, ol, scale=None, dtype="bf16", rows=None):
    out, lse = got
    n, hq, d = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    scale = d ** -0.5 if scale is None else scale
    errors, sizes = [], []
    for b in range(n) if rows is None else rows:
        g = b // (n // len(pt))
        where = []
        for table, length in ((pt[g], int(pl[g])), (ot[b], int(ol[b]))):
            at = torch.arange(max(length, 0), device="cuda")
            where.append((table.long()[at // page], at % page))
        pages, slots = (torch.cat(x) for x in zip(*where))
        if len(pages) == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        k, v = kc[pages, slots].double(), vc[pages, slots].double()
        s = torch.einsum("hgd,nhd->hgn", q[b].double().view(hk, hq // hk, d), k) * scale
        want_lse = torch.logsumexp(s, -1)
        p = torch.exp(s - want_lse[..., None])
        want = torch.einsum("hgn,nhd->hgd", p, v).flatten(0, 1)
        size = torch.einsum("hgn,nhd->hgd", p, v.abs()).flatten(0, 1)
        tol = UNIT[dtype] * want.abs() + (UNIT[dtype] + 2.0 ** -12) * size + 2.0 ** -25
        err = out[b].double() - want
        assert float((err.abs() - tol).max()) <= 0, (b, float((err.abs() - tol).max()))
        err_lse = (lse[b].double() - want_lse.flatten()).abs()
        assert float((err_lse - 2.0 ** -18 * (1 + want_lse.flatten().abs())).max()) <= 0, b
        errors.append(err)
        sizes.append(want)
    if errors:
        assert float(torch.stack(errors).norm()) <= 1.5 * UNIT[dtype] * float(torch.stack(sizes).norm())


SHAPES = [  # prefixes, own lengths, query heads, key heads, dim, page
    ([1025], [130, 0, 1, 64, 5, 77, 128, 9], 8, 1, 128, 16),
    ([1], [1], 1, 1, 64, 1), ([128], [0], 4, 4, 128, 128), ([129, 127], [3, 0, 500, 1], 6, 2, 96, 24),
    ([0, 2000], [20, 0, 0, 7], 8, 2, 128, 16), ([5000], list(range(0, 700, 10)), 16, 4, 64, 64),
    ([700, 64, 63, 0, 65], [11] * 15, 12, 12, 64, 24), ([3000], [100] * 40, 8, 1, 256, 16), ([900, 300], [40] * 34, 9, 3, 192, 7),
    ([20000], [300, 0, 17], 32, 8, 128, 64), ([260], [33] * 9, 64, 2, 256, 48), ([257], [1] * 130, 2, 1, 96, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("prefixes,own,hq,hk,d,page", SHAPES)
def test_attention(prefixes, own, hq, hk, d, page, dtype):
    a = build(prefixes, own, hq, hk, d, page, dtype)
    check(attend(*a), *a, dtype=dtype)


@pytest.mark.parametrize("layout", ["head", "pair"])
def test_cache_layouts(layout):
    a = build([333, 70], [5, 300, 77, 0], 8, 2, 128, 16, layout=layout)
    check(attend(*a), *a)


@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_scale_and_strided_queries(scale):
    a = build([500], [100, 1, 30], 8, 2, 128, 16)
    q, page = a[0], 16
    wide = torch.full((3, 12, 136), math.nan, device="cuda", dtype=torch.bfloat16)
    wide[:, 2:10, :128] = q
    out = torch.full((3, 9, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(3, 8, device="cuda")
    ws = dc.prefix_attention_workspace(3, 1, 8, 2, 128, a[3].shape[1] * page, a[5].shape[1] * page)
    dc.prefix_attention(wide[:, 2:10, :128], *a[1:], out[:, 1:], ws, scale=scale, lse=lse)
    check((out[:, 1:], lse), *a, scale=scale)
    assert bool((out[:, 0] == 5).all())


@pytest.mark.parametrize("d", [64, 128, 192])
def test_large_scores_that_move_the_reference(d):
    """Scores that grow along the prefix, one key far ahead late in it, and one among a sequence's own tokens."""
    a = build([4000], [200, 3, 0], 8, 2, d, 64)
    q, kc, vc, pt, pl, ot, ol = a
    q *= 4
    for i in range(4000 // 64):
        kc[pt[0, i].long()] *= 0.2 + i / 20
    kc[pt[0, 50].long(), 9] = q[0, ::4] * 2
    kc[ot[0, 1].long(), 5] = q[0, ::4] * 3
    check(attend(*a), *a)


@pytest.mark.parametrize("hq,hk,d", [(8, 1, 128), (32, 8, 64), (4, 2, 256)])
def test_bits_do_not_depend_on_the_batch(hq, hk, d):
    a = build([5000, 900], [300, 0, 1, 77, 128, 40] * 6, hq, hk, d, 16)
    q, kc, vc, pt, pl, ot, ol = a
    want = attend(*a)
    again = attend(*a)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    for b in (0, 1, 7, 17, 18, 35):
        g = b // 18
        one = attend(q[b:b + 1], kc, vc, pt[g:g + 1], pl[g:g + 1], ot[b:b + 1], ol[b:b + 1])
        assert torch.equal(one[0][0], want[0][b]) and torch.equal(one[1][0], want[1][b]), b
    # another place among other sequences, wider tables
    some = torch.tensor([17, 3, 0, 9, 5, 1], device="cuda")
    wide = torch.full((1, pt.shape[1] * 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :pt.shape[1]] = pt[:1]
    got = attend(q[some], kc, vc, wide, pl[:1], ot[some], ol[some])
    assert torch.equal(got[0], want[0][some]) and torch.equal(got[1], want[1][some])


def test_against_paged_attention_of_whole_sequences():
    """The same tokens as one context: both within their tolerances, lse to binary32."""
    a = build([640], [50, 0, 7, 100], 16, 4, 128, 16)
    q, kc, vc, pt, pl, ot, ol = a
    out, lse = attend(*a)
    table = torch.cat([pt.expand(4, -1)[:, :40], ot], 1).contiguous()
    lengths = ol + 640
    whole, whole_lse = torch.empty_like(out), torch.empty_like(lse)
    dc.paged_attention(q, kc, vc, table, lengths, whole, dc.attention_workspace(4, 16, 4, 128, table.shape[1] * 16), lse=whole_lse)
    assert float((lse - whole_lse).abs().max()) <= 2.0 ** -17 * (1 + float(lse.abs().max()))
    assert float((out.float() - whole.float()).norm()) <= 2 * UNIT["bf16"] * float(whole.float().norm())


def test_places_that_do_not_exist_give_nan():
    a = build([500, 500, 300, 100], [10, 20, 30, 0] * 2, 8, 2, 128, 16)
    q, kc, vc, pt, pl, ot, ol = a
    pt[0, 3] = kc.shape[0]       # group 0: sequences 0 and 1
    pl[1] = pt.shape[1] * 16 + 1  # group 1: 2 and 3
    ot[4, 0] = -1                # sequence 4 alone
    pl[3] = -7                   # group 3 has no prefix
    out, lse = attend(*a)
    for b in (0, 1, 2, 3, 4):
        assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
    check((out, lse), *a, rows=[5, 6, 7])
    assert bool((out[7] == 0).all())  # (its prefix is empty, and so are its own tokens)


def test_nan_and_infinity_of_attended_tokens():
    a = build([200], [40, 40, 0], 8, 1, 64, 16)
    q, kc, vc, pt, pl, ot, ol = a
    want = attend(*a)
    kc[ot[0, 1].long(), 3] = math.nan  # one sequence's own
    got = attend(*a)
    assert bool(torch.isnan(got[0][0]).all()) and torch.equal(got[0][1:], want[0][1:])
    vc[pt[0, 2].long(), 5, 0, 9] = math.inf  # everyone's
    got = attend(*a)
    assert not bool(torch.isfinite(got[0][:, :, 9]).any())
    keep = [i for i in range(64) if i != 9]
    assert torch.equal(got[0][1:][:, :, keep], want[0][1:][:, :, keep])


def test_offsets_past_32_bits():
    pages, page, hk, d = 70000, 64, 4, 128  # 2.3e9 elements
    kc = torch.empty(pages, page, hk, d, device="cuda", dtype=torch.bfloat16)
    vc = torch.empty_like(kc)
    pt = torch.tensor([[69999, 3, 65536]], dtype=torch.int32, device="cuda")
    ot = torch.tensor([[40000], [69998]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in (69999, 3, 65536, 40000, 69998):
        kc[i], vc[i] = (torch.randn(page, hk, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, 8, d, generator=g, device="cuda").to(torch.bfloat16)
    a = q, kc, vc, pt, torch.tensor([190], dtype=torch.int32, device="cuda"), ot, torch.tensor([64, 9], dtype=torch.int32, device="cuda")
    check(attend(*a), *a)


def test_one_workspace_for_many_calls():
    ws = dc.prefix_attention_workspace(24, 4, 32, 8, 256, 5000, 3000)
    for prefixes, own, hq, hk, d, page in (([4990], [2990] * 4, 8, 2, 128, 16), ([300, 20], [9, 0, 77, 1], 16, 2, 64, 16),
                                           ([4000] * 4, [600] * 24, 32, 8, 64, 64), ([4990], [2990] * 4, 8, 2, 128, 16)):
        a = build(prefixes, own, hq, hk, d, page)
        for _ in range(2):
            check(attend(*a, workspace=ws), *a)


def test_streams_graphs_and_versions():
    a = build([3000, 100], [17, 900, 0, 40], 16, 2, 128, 16)
    want = attend(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attend(*a, stream=side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = dc.prefix_attention_workspace(4, 2, 16, 2, 128, a[3].shape[1] * 16, a[5].shape[1] * 16)
    before = out._version, lse._version
    dc.prefix_attention(*a, out, ws, lse=lse)
    assert out._version > before[0] and lse._version > before[1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dc.prefix_attention(*a, out, ws, lse=lse)
    for _ in range(3):
        out.fill_(3)
        lse.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # lengths and tables are read on the GPU: a replay follows them
    a[6][1] = 600
    graph.replay()
    torch.cuda.synchronize()
    check((out, lse), *a)


@pytest.mark.parametrize("prefixes,own", [([900, 40], [0, 300, 7, 64]), ([0, 3000], [0, 0, 1, 2])])
def test_follows_the_calls_before_and_after_it(prefixes, own):
    """Calls without a wait between them: appends write both parts' slots and the queries, each attention reads them,
    and the next append overwrites them."""
    hq, hk, d, page = 16, 2, 128, 16
    q, kc, vc, pt, pl, ot, ol = build(prefixes, own, hq, hk, d, page)
    tables = torch.full((6, max(pt.shape[1], ot.shape[1])), -1, dtype=torch.int32, device="cuda")
    tables[:2, :pt.shape[1]] = pt
    tables[2:, :ot.shape[1]] = ot
    where = [(s, t) for s, n in enumerate(prefixes + own) for t in sorted({0, n // 2, n - 1}) if n > 0]  # (a slot once)
    seqs, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*where))
    steps = 12
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(steps, len(where), hk, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    new = torch.randn(steps, *q.shape, generator=g, device="cuda").to(torch.bfloat16)
    ws = dc.prefix_attention_workspace(4, 2, hq, hk, d, pt.shape[1] * page, ot.shape[1] * page)
    results = []
    for wait in (True, False):
        out = torch.zeros(steps, *q.shape, device="cuda", dtype=q.dtype)
        torch.cuda.synchronize()
        for i in range(steps):
            dc.kv_append(k[i], v[i], pos, seqs, tables, kc, vc)
            q.copy_(new[i])
            if wait:
                torch.cuda.synchronize()
            dc.prefix_attention(q, kc, vc, pt, pl, ot, ol, out[i], ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(out)
    assert torch.equal(*results)


@pytest.mark.parametrize("page", [16, 7])
def test_tables_and_lengths_that_change_between_calls(page):
    """... without a wait: each call reads the tables, lengths, keys and values that were written just before it."""
    hq, hk, d, steps = 8, 2, 128, 16
    q, kc, vc, pt, pl, ot, ol = build([900, 300], [200, 0, 7, 64], hq, hk, d, page)
    g = torch.Generator(device="cuda").manual_seed(10)
    held = torch.cat([t[t >= 0] for t in (pt, ot)])
    kc.nan_to_num_(0.0)
    vc.nan_to_num_(0.0)
    pick = lambda t: held[torch.randint(0, len(held), t.shape, generator=g, device="cuda")]
    tables = [(pick(pt), pick(ot)) for _ in range(steps)]
    lengths = [tuple(torch.randint(0, t.shape[1] * page + 1, (len(t),), generator=g, device="cuda").int() for t in (pt, ot)) for _ in range(steps)]
    new = torch.randn(steps, 5, hk, d, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(5, dtype=torch.int32, device="cuda") * page
    zero = torch.zeros(5, dtype=torch.int32, device="cuda")
    where = torch.stack([held[torch.randperm(len(held), generator=g, device="cuda")[:5]] for _ in range(steps)])  # (a slot once a call)
    caches = kc.clone(), vc.clone()
    ws = dc.prefix_attention_workspace(4, 2, hq, hk, d, pt.shape[1] * page, ot.shape[1] * page)
    results = []
    for wait in (True, False):
        out, lse = torch.zeros(steps, *q.shape, device="cuda", dtype=q.dtype), torch.zeros(steps, 4, hq, device="cuda")
        kc.copy_(caches[0])
        vc.copy_(caches[1])
        torch.cuda.synchronize()
        for i in range(steps):
            for to, have in zip((pt, ot, pl, ol), (*tables[i], *lengths[i])):
                to.copy_(have)
            dc.kv_append(new[i], new[i], pos, zero, where[i:i + 1], kc, vc)
            if wait:
                torch.cuda.synchronize()
            dc.prefix_attention(q, kc, vc, pt, pl, ot, ol, out[i], ws, lse=lse[i])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append((out, lse))
    check((results[0][0][-1], results[0][1][-1]), q, kc, vc, pt, pl, ot, ol)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


def test_sums_over_long_prefixes_are_cut():
    """Flat scores and positive values of a million tokens, few CTAs a key head (the tokens' pages come again and
    again).  Weights are 1, so the output is off by its last rounding (2^-11), and by sums of at most 24576 tokens on
    the tensor cores, 16 at a time, each cut rather than rounded at worst (1536 times 2^-23); 2^-15 for the others."""
    tokens, hk, d, page = 1 << 20, 32, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.randn(9, page, hk, d, generator=g, device="cuda").half()
    vc = (1 + torch.rand(9, page, hk, d, generator=g, device="cuda")).half()
    pt = (torch.arange(tokens // page, device="cuda") % 8).int()[None]
    q = torch.zeros(2, hk, d, device="cuda", dtype=torch.float16)
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = attend(q, kc, vc, pt, one(tokens), one(8, 8)[:, None], one(0, 1))
    want = vc[:8].double().mean((0, 1))
    for b in range(2):
        assert float(((out[b].double() - want).abs() / want).max()) <= 2.0 ** -11 + 1536 * 2.0 ** -23 + 2.0 ** -15
        assert float((lse[b] - math.log(tokens + b)).abs().max()) <= 2.0 ** -18 * (1 + math.log(tokens))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hk,tokens", [(1, 1 << 22), (160, 1 << 15)])
def test_more_chunks_than_fill_the_gpu(hk, tokens, dtype):
    """(Pages that come again and again: the softmax is that over each once.)"""
    d, page, pages = 64, 64, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.randn(pages + 1, page, hk, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    pt = (torch.arange(tokens // page, device="cuda") % pages).int()[None]
    q = torch.randn(2, hk, d, generator=g, device="cuda").to(DT[dtype])
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = attend(q, kc, vc, pt, one(tokens), one(8, 8)[:, None], one(0, 0))
    again = torch.log(torch.tensor(tokens // (page * pages), dtype=torch.float64))
    table = torch.arange(pages, device="cuda").int()[None]
    check((out, (lse.double() - again.item()).float()), q, kc, vc, table, one(pages * page), one(8, 8)[:, None], one(0, 0), dtype=dtype)


def test_a_chunk_at_a_time_of_many_key_heads():
    a = build([50000, 24577], [30, 0], 80, 80, 64, 64, "f16")
    check(attend(*a), *a, dtype="f16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [2.0 ** 12, 2.0 ** 16, 2.0 ** 20, 2.0 ** 27, -2.0 ** 33, 2.0 ** 33])
def test_scores_of_which_only_the_largest_count(scale, dtype):
    """Whole numbers, so that the scores are exact: tokens with the largest share the weight evenly.  (Scores of 2^39
    are as far as the reference's lse holds the log of how many they are.)"""
    a = build([2000, 700], [50, 0, 7, 300], 8, 2, 64, 16, dtype)
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in (a[0], a[1]):
        t.copy_(torch.randint(-2, 3, t.shape, generator=g, device="cuda").to(t.dtype))
    check(attend(*a, scale=scale), *a, scale=scale, dtype=dtype)
