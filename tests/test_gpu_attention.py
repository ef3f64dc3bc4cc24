"""kv_append and paged_attention against the formulas in 64 bits.

Tolerances, from the arithmetic.  Attention: one rounding of the output to 16
bits; scores are sums of dim products in binary32 (2^-24 of sum |q||k| a few
times over), weights carry 2^-17 (a pair of 16-bit numbers) and the
exponential's 2^-22, so the output is within 2^-13 of sum p |v| besides its
rounding.  The cache: two products and a sum in binary32 and one rounding.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import reduce_copy_rank_gb300 as dc  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LENGTHS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4099, 8193]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)


def build(lengths, hq, hk, d, page, dtype="bf16", seed=0, layout="token", spare=2, poison=True):
    """Queries, caches (slots that hold no token are NaN), table (-1 past the end), lengths."""
    g = torch.Generator(device="cuda").manual_seed(seed + 17)
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if layout == "token":
        kc, vc = (torch.randn(pages, page, hk, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    elif layout == "head":  # heads outside tokens
        kc, vc = (torch.randn(pages, hk, page, d, generator=g, device="cuda").to(DT[dtype]).transpose(1, 2) for _ in range(2))
    else:  # keys and values of a page side by side in one tensor
        both = torch.randn(pages, 2, page, hk, d, generator=g, device="cuda").to(DT[dtype])
        kc, vc = both[:, 0], both[:, 1]
    if poison:
        held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lengths):
            for i in range(need[b]):
                held[table[b, i].long(), :min(page, n - i * page)] = True
        kc[~held] = math.nan
        vc[~held] = math.nan
    q = torch.randn(len(lengths), hq, d, generator=g, device="cuda").to(DT[dtype])
    return q, kc, vc, table, torch.tensor(lengths, dtype=torch.int32, device="cuda")


def attend(q, kc, vc, table, lengths, window=0, scale=None, workspace=None, stream=None):
    n, hq, d = q.shape
    if workspace is None:
        workspace = dc.attention_workspace(n, hq, kc.shape[2], d, table.shape[1] * kc.shape[1])
    out = torch.full((n, hq, d), 7.0, device="cuda", dtype=q.dtype)
    lse = torch.full((n, hq), 7.0, device="cuda")
    assert dc.paged_attention(q, kc, vc, table, lengths, out, workspace, scale=scale, window=window, lse=lse,
                              stream=stream) is out
    torch.cuda.synchronize()
    return out, lse


def check(got, q, kc, vc, table, lengths, window=0, scale=None, dtype="bf16"):
    out, lse = got
    n, hq, d = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    scale = d ** -0.5 if scale is None else scale
    for b, length in enumerate(lengths.tolist()):
        start = max(0, length - window) if window else 0
        if length == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        at = torch.arange(start, length, device="cuda")
        rows = table[b].long()[at // page], at % page
        k, v = kc[rows].double(), vc[rows].double()
        s = torch.einsum("hgd,nhd->hgn", q[b].double().view(hk, hq // hk, d), k) * scale
        want_lse = torch.logsumexp(s, -1)
        p = torch.exp(s - want_lse[..., None])
        want = torch.einsum("hgn,nhd->hgd", p, v).flatten(0, 1)
        size = torch.einsum("hgn,nhd->hgd", p, v.abs()).flatten(0, 1)
        tol = UNIT[dtype] * want.abs() + 2.0 ** -13 * size + 2.0 ** -25
        over = (out[b].double() - want).abs() - tol
        assert float(over.max()) <= 0, (b, length, float(over.max()))
        err = (lse[b].double() - want_lse.flatten()).abs()
        assert float((err - 2.0 ** -18 * (1 + want_lse.flatten().abs())).max()) <= 0, (b, length)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hk,d,page", [
    (8, 1, 128, 16), (4, 4, 64, 1), (3, 1, 64, 24), (10, 2, 96, 64), (32, 2, 128, 16), (9, 1, 64, 128), (17, 1, 128, 32),
    (64, 2, 256, 16), (7, 1, 192, 48), (6, 2, 256, 7), (12, 1, 96, 16), (16, 1, 192, 64)])
def test_attention(dtype, hq, hk, d, page):
    a = build(LENGTHS, hq, hk, d, page, dtype)
    check(attend(*a), *a, dtype=dtype)


@pytest.mark.parametrize("layout", ["head", "pair"])
def test_cache_layouts(layout):
    a = build([5, 300, 77], 8, 2, 128, 16, layout=layout)
    check(attend(*a), *a)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 1000, 5000])
def test_window(window):
    a = build(LENGTHS, 8, 2, 64, 16, "f16")
    check(attend(*a, window=window), *a, window=window, dtype="f16")


def test_window_reads_nothing_before_it():
    a = build([500, 40], 4, 1, 128, 16)
    q, kc, vc, table, lengths = a
    want = attend(*a, window=30)
    table[0, :(500 - 30) // 16] = -1  # pages already given back
    got = attend(*a, window=30)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_scale_and_strided_queries():
    q, kc, vc, table, lengths = build([100, 1, 700], 8, 2, 128, 16)
    wide = torch.full((3, 12, 136), math.nan, device="cuda", dtype=torch.bfloat16)
    wide[:, 2:10, :128] = q
    view = wide[:, 2:10, :128]
    out = torch.full((3, 9, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(3, 8, device="cuda")
    ws = dc.attention_workspace(3, 8, 2, 128, table.shape[1] * 16)
    dc.paged_attention(view, kc, vc, table, lengths, out[:, 1:], ws, scale=0.3, lse=lse)
    check((out[:, 1:], lse), q, kc, vc, table, lengths, scale=0.3)
    assert bool((out[:, 0] == 5).all())


def test_long_and_large_scores():
    """A long sequence of many pieces, and scores that need the running maximum."""
    q, kc, vc, table, lengths = build([70001, 3], 8, 1, 64, 64, spare=1)
    q *= 8
    check(attend(q, kc, vc, table, lengths), q, kc, vc, table, lengths)
    kc[table[0, 1000].long(), 5] = q[0, :1] * 2  # one key far ahead of the rest
    check(attend(q, kc, vc, table, lengths), q, kc, vc, table, lengths)


@pytest.mark.parametrize("hq,hk,d", [(8, 1, 128), (32, 8, 64)])
def test_bits_do_not_depend_on_the_batch(hq, hk, d):
    a = build([9000, 0, 130, 4000, 1, 2500], hq, hk, d, 16)
    q, kc, vc, table, lengths = a
    want = attend(*a)
    again = attend(*a)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    for b in range(len(lengths)):
        one = attend(q[b:b + 1], kc, vc, table[b:b + 1], lengths[b:b + 1])
        assert torch.equal(one[0][0], want[0][b]) and torch.equal(one[1][0], want[1][b]), b
        # nor on how wide the table is
        wide = torch.full((1, table.shape[1] * 3), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table[b]
        one = attend(q[b:b + 1], kc, vc, wide, lengths[b:b + 1])
        assert torch.equal(one[0][0], want[0][b]), b


def test_one_workspace_for_calls_of_every_shape():
    ws = dc.attention_workspace(6, 32, 8, 128, 6000)
    for lengths, hq, hk, d, page in (([6000] * 6, 32, 8, 128, 16), ([3000], 8, 1, 64, 16), ([1, 2], 16, 1, 128, 16),
                                     ([5000, 200, 3], 32, 8, 128, 64), ([6000] * 6, 32, 8, 128, 16)):
        a = build(lengths, hq, hk, d, page)
        for _ in range(2):
            check(attend(*a, workspace=ws), *a)


def test_places_that_do_not_exist_give_nan():
    q, kc, vc, table, lengths = build([500, 500, 33, 40, 100, 20], 8, 2, 128, 16)
    pages = kc.shape[0]
    table[0, 3] = pages
    table[1, 30] = -1
    table[2, 2] = 2 ** 31 - 1
    lengths[3] = table.shape[1] * 16 + 1
    lengths[4] = -5
    out, lse = attend(q, kc, vc, table, lengths)
    for b in range(4):
        assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
    assert bool((out[4] == 0).all()) and bool((lse[4] == -math.inf).all())
    check((out[5:], lse[5:]), q[5:], kc, vc, table[5:], lengths[5:])


def test_nan_and_infinity_of_attended_tokens():
    q, kc, vc, table, lengths = build([40, 40, 40], 8, 1, 64, 16)
    kc[table[0, 1].long(), 3] = math.nan
    vc[table[1, 1].long(), 3, 0, 7] = math.inf
    out, lse = attend(q, kc, vc, table, lengths)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert bool((out[1, :, 7] == math.inf).all())
    keep = [i for i in range(64) if i != 7]
    assert bool(torch.isfinite(out[1][:, keep]).all())
    check((out[2:], lse[2:]), q[2:], kc, vc, table[2:], lengths[2:])


def test_cache_offsets_past_32_bits():
    pages, page, hk, d = 70000, 64, 4, 128  # 2.3e9 elements
    kc = torch.empty(pages, page, hk, d, device="cuda", dtype=torch.bfloat16)
    vc = torch.empty_like(kc)
    table = torch.tensor([[69999, 3, 65536], [40000, 69998, 0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([190, 129], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 319
    k, v, q = (torch.randn(n, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hk, hk, 8))
    seqs = torch.tensor([0] * 190 + [1] * 129, dtype=torch.int32, device="cuda")
    pos = torch.tensor([*range(190), *range(129)], dtype=torch.int32, device="cuda")
    dc.kv_append(k, v, pos, seqs, table, kc, vc)
    assert torch.equal(kc[69999, 5], k[5]) and torch.equal(vc[0, 0], v[190 + 128])
    a = (q[:2], kc, vc, table, lengths)
    check(attend(*a), *a)


def test_streams_and_graphs():
    a = build([3000, 17, 900], 16, 2, 128, 16)
    q, kc, vc, table, lengths = a
    want = attend(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attend(*a, stream=side)
    assert torch.equal(got[0], want[0])
    out = torch.empty_like(q)
    ws = dc.attention_workspace(3, 16, 2, 128, table.shape[1] * 16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dc.paged_attention(q, kc, vc, table, lengths, out, ws)
    lengths[0] = 2000
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, attend(*a)[0])


def test_attention_refusals():
    q, kc, vc, table, lengths = build([500, 3], 8, 2, 128, 16)
    ws = dc.attention_workspace(2, 8, 2, 128, table.shape[1] * 16)
    out = torch.empty_like(q)
    bad = [
        (ValueError, lambda: dc.paged_attention(q.float(), kc, vc, table, lengths, out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc.half(), vc, table, lengths, out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc, vc[:-1], table, lengths, out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc, vc, table.long(), lengths, out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc, vc, table, lengths.long(), out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc, vc, table[:1], lengths, out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc, vc, table, lengths, out[:, :4], ws)),
        (ValueError, lambda: dc.paged_attention(q.cpu(), kc, vc, table, lengths, out, ws)),
        (ValueError, lambda: dc.paged_attention(q, kc, vc, table, lengths, out, ws.cpu())),
        (ValueError, lambda: dc.paged_attention(q[..., :64], kc, vc, table, lengths, out[..., :64], ws)),
        (dc.DCError, lambda: dc.paged_attention(q, kc, vc, table, lengths, out, ws[:256])),
        (dc.DCError, lambda: dc.paged_attention(q, kc, vc, table, lengths, q, ws)),
        (dc.DCError, lambda: dc.paged_attention(q, kc, vc, table, lengths, out, ws, window=-1)),
        (dc.DCError, lambda: dc.paged_attention(q[:, :7], kc, vc, table, lengths, out[:, :7], ws)),
        (dc.DCError, lambda: dc.paged_attention(q, kc, vc, table, lengths, out, ws, scale=math.inf)),
        (dc.DCError, lambda: dc.paged_attention(q[..., :80].contiguous(), kc[..., :80], vc[..., :80], table, lengths,
                                                out[..., :80].contiguous(), ws)),
        (dc.DCError, lambda: dc.attention_workspace(2, 8, 3, 128, 100)),
        (dc.DCError, lambda: dc.attention_workspace(2, 8, 2, 80, 100)),
    ]
    before = dc.launch_count()
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was not refused")
    assert dc.launch_count() == before
    dc.paged_attention(q[:0], kc, vc, table[:0], lengths[:0], out[:0], ws)
    assert dc.launch_count() == before


# ---------------------------------------------------------------- the cache
def angles(rows, rot, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    a = torch.rand(rows, rot // 2, generator=g, device="cuda") * 6.3
    return torch.cat([a.cos(), a.sin()], 1).contiguous()


def rotated(x, cs, rot, interleaved):
    """The rotation in 64 bits, and the size of its terms."""
    x, cs = x.double(), cs.double()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    out, size = x.clone(), x.abs().clone()
    a_at = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    b_at = a_at + 1 if interleaved else a_at + rot // 2
    a, b = x[..., a_at], x[..., b_at]
    out[..., a_at], out[..., b_at] = a * c - b * s, b * c + a * s
    size[..., a_at] = size[..., b_at] = a.abs() + b.abs()
    return out, size


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,interleaved,page", [
    (1, 8, 1, 128, 128, False, 16), (7, 4, 4, 64, 32, False, 1), (33, 32, 8, 128, 128, True, 64), (300, 6, 2, 80, 32, True, 24),
    (5, 0, 3, 8, 0, False, 16), (513, 16, 16, 96, 96, False, 16), (64, 3, 1, 256, 64, False, 128), (2, 1, 1, 1024, 1024, False, 2),
    (2, 64, 8, 16, 16, True, 5), (3, 2, 1, 1024, 0, False, 4), (9, 1, 2, 1024, 512, True, 4)])
def test_append(dtype, tokens, hq, hk, d, rot, interleaved, page):
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(tokens)
    B = min(tokens, 5)
    seqs = torch.arange(tokens, device="cuda", dtype=torch.int32) % B
    pos = torch.arange(tokens, device="cuda", dtype=torch.int32) // B + 3 * seqs
    width = int(pos.max()) // page + 2
    pages = B * width + 1
    table = torch.randperm(pages, generator=g, device="cuda")[:B * width].int().view(B, width)
    both = torch.randn(tokens, hq + 2 * hk, d, generator=g, device="cuda").to(dt)
    q, k, v = both[:, :hq], both[:, hq:hq + hk], both[:, hq + hk:]
    kc, vc = (torch.full((pages, page, hk, d), 9.0, device="cuda", dtype=dt) for _ in range(2))
    cs = angles(int(pos.max()) + 1, rot) if rot else None
    out = torch.empty(tokens, hq, d, device="cuda", dtype=dt) if hq else None
    dc.kv_append(k, v, pos, seqs, table, kc, vc, q=q if hq else None, q_out=out, cos_sin=cs, interleaved=interleaved)
    torch.cuda.synchronize()
    page_of = table[seqs.long(), pos.long() // page].long()
    held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    held[page_of, pos.long() % page] = True
    assert int(held.sum()) == tokens
    assert bool((kc[~held] == 9).all()) and bool((vc[~held] == 9).all())
    assert torch.equal(vc[page_of, pos.long() % page], v)
    for got, x in ((kc[page_of, pos.long() % page], k), (out, q)):
        if got is None:
            continue
        if rot == 0:
            assert torch.equal(got, x)
            continue
        want, size = rotated(x, cs[pos.long()], rot, interleaved)
        # three roundings in binary32, one to the type
        over = (got.double() - want).abs() - (UNIT[dtype] * want.abs() + 2.0 ** -22 * size + (2.0 ** -25 if dtype == "f16" else 0))
        assert float(over.max()) <= 0
        assert torch.equal(got[..., rot:], x[..., rot:])
    if hq:  # in place
        dc.kv_append(k, v, pos, seqs, table, kc, vc, q=q, q_out=q, cos_sin=cs, interleaved=interleaved)
        assert torch.equal(q, out)


def test_append_padding_and_places_that_do_not_exist():
    page, hk, d = 16, 2, 64
    table = torch.tensor([[0, 5], [2, 9]], dtype=torch.int32, device="cuda")  # page 9 does not exist
    kc, vc = (torch.full((6, page, hk, d), 9.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v, q = (torch.randn(8, hk, d, device="cuda").to(torch.bfloat16) for _ in range(3))
    out = torch.full_like(q, 5.0)
    pos = torch.tensor([0, -1, 31, 32, 16, 3, 3, 29], dtype=torch.int32, device="cuda")
    seqs = torch.tensor([0, 0, 0, 0, 1, 2, -1, 0], dtype=torch.int32, device="cuda")
    cs = angles(30, d)  # position 31 has no angles
    dc.kv_append(k, v, pos, seqs, table, kc, vc, q=q, q_out=out, cos_sin=cs)
    torch.cuda.synchronize()
    held = torch.zeros(6, page, dtype=torch.bool, device="cuda")
    held[0, 0] = held[5, 13] = True
    assert bool((kc[~held] == 9).all()) and bool((vc[~held] == 9).all())
    assert torch.equal(vc[0, 0], v[0]) and torch.equal(vc[5, 13], v[7])
    assert bool((out[1] == 5).all())
    for i in (2, 3, 4, 5, 6):
        assert bool(torch.isnan(out[i]).all()), i
    assert bool(torch.isfinite(out[[0, 7]]).all())


def test_append_then_attend_step_by_step():
    """A sequence grown one token at a time attends as one written at once."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n, hq, hk, d, page = 70, 8, 2, 64, 16
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(torch.float16) for h in (hq, hk, hk))
    table = torch.arange(8, device="cuda", dtype=torch.int32)[None]
    cs = angles(n, d)
    kc, vc = (torch.full((8, page, hk, d), math.nan, device="cuda", dtype=torch.float16) for _ in range(2))
    ws = dc.attention_workspace(1, hq, hk, d, 128)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    for t in range(n):
        pos = torch.tensor([t], dtype=torch.int32, device="cuda")
        qr = torch.empty_like(q[:1])
        dc.kv_append(k[t:t + 1], v[t:t + 1], pos, zero, table, kc, vc, q=q[t:t + 1], q_out=qr, cos_sin=cs)
        outs.append(dc.paged_attention(qr, kc, vc, table, pos + 1, torch.empty_like(qr), ws))
    kc2, vc2 = torch.full_like(kc, math.nan), torch.full_like(vc, math.nan)
    all_pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qr = torch.empty_like(q)
    dc.kv_append(k, v, all_pos, torch.zeros_like(all_pos), table, kc2, vc2, q=q, q_out=qr, cos_sin=cs)
    at_once = dc.paged_attention(qr, kc2, vc2, table.expand(n, 8).contiguous(), all_pos + 1, torch.empty_like(q),
                                 dc.attention_workspace(n, hq, hk, d, 128))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(outs), at_once)


def test_append_refusals():
    k = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    v = k.clone()
    pos, seqs = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cs = angles(64, 64)
    odd = torch.zeros(4, 2, 65, device="cuda", dtype=torch.bfloat16)
    bad = [
        (ValueError, lambda: dc.kv_append(k.cpu(), v, pos, seqs, table, kc, vc)),
        (ValueError, lambda: dc.kv_append(k, v[:3], pos, seqs, table, kc, vc)),
        (ValueError, lambda: dc.kv_append(k, v.float(), pos, seqs, table, kc, vc)),
        (ValueError, lambda: dc.kv_append(k, v, pos.long(), seqs, table, kc, vc)),
        (ValueError, lambda: dc.kv_append(k, v, pos, seqs[:2], table, kc, vc)),
        (ValueError, lambda: dc.kv_append(k, v, pos, seqs, table, kc[..., :32], vc[..., :32])),
        (ValueError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc[:2])),
        (ValueError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc, q=k)),
        (ValueError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc, q_out=k)),
        (ValueError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc, cos_sin=cs.half())),
        (dc.DCError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, kc)),
        (dc.DCError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc, cos_sin=angles(64, 24))),
        (dc.DCError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc, cos_sin=angles(64, 128))),
        (dc.DCError, lambda: dc.kv_append(odd[..., :64], v, pos, seqs, table, kc, vc)),
        (dc.DCError, lambda: dc.kv_append(odd[..., 1:], v, pos, seqs, table, kc, vc)),
        (dc.DCError, lambda: dc.kv_append(k, v, pos, seqs, table, kc, vc, q=v, q_out=k)),
        (dc.DCError, lambda: dc.kv_append(kc[0, :4], v, pos, seqs, table, kc, vc)),
    ]
    before = dc.launch_count()
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was not refused")
    assert dc.launch_count() == before
    dc.kv_append(k[:0], v[:0], pos[:0], seqs[:0], table, kc, vc)
    assert dc.launch_count() == before


def test_one_long_sequence_among_short_ones():
    """Many sequences and one far longer."""
    lengths = [70001] + [40 + 7 * b for b in range(39)]
    q, kc, vc, table, lengths = build(lengths, 8, 8, 64, 64, "f16", spare=1)
    got = attend(q, kc, vc, table, lengths)
    check(got, q, kc, vc, table, lengths, dtype="f16")
    one = attend(q[:1], kc, vc, table[:1], lengths[:1])
    assert torch.equal(got[0][:1], one[0]) and torch.equal(got[1][:1], one[1])


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (8, 2, 128), (16, 1, 128), (6, 2, 192), (32, 1, 256), (6, 2, 96)])
def test_bits_do_not_depend_on_the_grid(hq, hk, d):
    """A sequence alone (pieces joined in a cluster or by the last to finish),
    in a small batch and in one that fills the GPU several times."""
    q, kc, vc, table, lengths = build([3000, 700, 257, 5000, 64, 9000], hq, hk, d, 16)
    want = attend(q, kc, vc, table, lengths)
    for copies in (2, 9, 60):
        many = attend(q.repeat(copies, 1, 1), kc, vc, table.repeat(copies, 1), lengths.repeat(copies))
        for i in (0, copies - 1):
            assert torch.equal(many[0][6 * i:6 * i + 6], want[0]) and torch.equal(many[1][6 * i:6 * i + 6], want[1]), copies
    for b in range(6):
        one = attend(q[b:b + 1], kc, vc, table[b:b + 1], lengths[b:b + 1])
        assert torch.equal(one[0][0], want[0][b]) and torch.equal(one[1][0], want[1][b]), b


@pytest.mark.parametrize("hq,hk,d", [(9, 1, 64), (32, 2, 64), (12, 1, 96), (20, 1, 128), (64, 4, 128), (11, 1, 192), (48, 3, 256)])
def test_bits_of_large_groups_do_not_depend_on_the_grid(hq, hk, d):
    """More than 8 query heads a key head: alone a sequence's heads are split over CTAs, in a batch not."""
    q, kc, vc, table, lengths = build([1500, 33, 5, 260], hq, hk, d, 16)
    kc[2, 3, 0, :5] = 40.0
    vc[1, 2, 0, :7] = float("inf")
    want = attend(q, kc, vc, table, lengths)
    many = attend(q.repeat(80, 1, 1), kc, vc, table.repeat(80, 1), lengths.repeat(80))
    for i in (0, 79):
        for k in (0, 1):
            a, b = many[k][4 * i:4 * i + 4], want[k]
            bits = torch.int16 if k == 0 else torch.int32
            assert torch.equal(a.view(bits), b.view(bits))
    for b in range(4):
        one = attend(q[b:b + 1], kc, vc, table[b:b + 1], lengths[b:b + 1])
        assert torch.equal(one[0][0].view(torch.int16), want[0][b].view(torch.int16)) and torch.equal(one[1][0], want[1][b]), b


@pytest.mark.parametrize("seqs,hk", [(1, 1), (3, 8), (40, 8)])
def test_tables_far_wider_than_the_sequences(seqs, hk):
    lengths = [(b * 337) % 2900 for b in range(seqs)]
    lengths[0] = 1500
    q, kc, vc, table, lengths = build(lengths, 2 * hk, hk, 64, 16)
    want = attend(q, kc, vc, table, lengths)
    check(want, q, kc, vc, table, lengths)
    wide = torch.full((seqs, 8192), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    got = attend(q, kc, vc, wide, lengths)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (8, 1, 128), (6, 2, 192), (12, 1, 96), (16, 1, 64), (32, 2, 256)])
@pytest.mark.parametrize("copies", [1, 60])
def test_one_token_far_ahead_of_the_others(dtype, hq, hk, d, copies):
    """A token of value 0 whose score is far above all others': what is left of
    them is the result, and it carries the output's rounding alone."""
    cases = [(n, gap, size) for n in (17, 32, 100, 700) for gap, size in (
        (3.0, 1.0), (8.3, 1.0), (10.2, 20.0), (12.9, 900.0), (16.6, 5000.0), (20.3, 60000.0), (24.7, 60000.0))]
    q, kc, vc, table, lengths = build([c[0] for c in cases], hq, hk, d, 16, dtype)
    held = torch.isfinite(vc[..., :1])
    g = torch.Generator(device="cuda").manual_seed(9)
    near = torch.rand(kc.shape[:3], generator=g, device="cuda")
    kc[..., 0], kc[..., 1], kc[..., 2:] = 0.0, near.to(DT[dtype]), 0.0
    vc.copy_(torch.rand(vc.shape, generator=g, device="cuda") + 0.5)
    for b, (n, gap, size) in enumerate(cases):
        pages = table[b, :-(-n // 16)].long()
        vc[pages] = (vc[pages].float() * size / 1.5).to(DT[dtype])
        first = (n * 7) // 11
        kc[pages[first // 16], first % 16, :, 0] = gap
        vc[pages[first // 16], first % 16] = 0.0
    kc.masked_fill_(~held, math.nan)
    vc.masked_fill_(~held, math.nan)
    q.zero_()
    q[..., 0] = q[..., 1] = 1.0
    many = attend(q.repeat(copies, 1, 1), kc, vc, table.repeat(copies, 1), lengths.repeat(copies), scale=1.0)
    n = len(cases)
    check((many[0][-n:], many[1][-n:]), q, kc, vc, table, lengths, scale=1.0, dtype=dtype)


def test_long_and_large_scores_of_binary16():
    q, kc, vc, table, lengths = build([70001, 3], 8, 1, 64, 64, "f16", spare=1)
    q *= 8
    check(attend(q, kc, vc, table, lengths), q, kc, vc, table, lengths, dtype="f16")
    kc[table[0, 1000].long(), 5] = q[0, :1] * 2  # one key far ahead of the rest
    check(attend(q, kc, vc, table, lengths), q, kc, vc, table, lengths, dtype="f16")


@pytest.mark.parametrize("hq", [8, 16])
def test_nan_and_infinity_of_attended_tokens_of_binary16(hq):
    q, kc, vc, table, lengths = build([40, 40, 40], hq, 1, 64, 16, "f16")
    kc[table[0, 1].long(), 3] = math.nan
    vc[table[1, 1].long(), 3, 0, 7] = math.inf
    out, lse = attend(q, kc, vc, table, lengths)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert bool((out[1, :, 7] == math.inf).all())
    keep = [i for i in range(64) if i != 7]
    assert bool(torch.isfinite(out[1][:, keep]).all())
    check((out[2:], lse[2:]), q[2:], kc, vc, table[2:], lengths[2:], dtype="f16")


def test_one_buffer_passed_in_parts_of_different_lengths():
    """Calls that pass as much of a workspace as they need: a small one's partial results are no counters of a larger one."""
    small, large = dc.dc_attention_workspace_bytes(4, 8, 1, 128, 4096), dc.dc_attention_workspace_bytes(64, 32, 8, 128, 8192)
    assert small < large
    ws = torch.zeros(large, dtype=torch.uint8, device="cuda")
    a = build([4096, 3000, 17, 4000], 8, 1, 128, 64, spare=1)
    b = build([8192 - 37 * i for i in range(64)], 32, 8, 128, 64, spare=1)
    want_a, want_b = attend(*a), attend(*b)
    for _ in range(2):
        got = attend(*a, workspace=ws[:small])
        assert torch.equal(got[0], want_a[0]) and torch.equal(got[1], want_a[1])
        got = attend(*b, workspace=ws)
        assert torch.equal(got[0], want_b[0]) and torch.equal(got[1], want_b[1])


def test_more_sequences_than_counters():
    """So many sequences and key heads that a CTA computes each from end to end."""
    hk, d, page, pages = 64, 64, 1024, 129
    lengths = [131072, 70001, 9000, 700, 0, 1, 130] + [(b * 37) % 200 for b in range(1363)]
    g = torch.Generator(device="cuda").manual_seed(6)
    kc, vc = (torch.randn(pages, page, hk, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randint(0, pages, (len(lengths), 128), generator=g, device="cuda", dtype=torch.int32)
    table[0] = torch.arange(128, 0, -1)
    q = torch.randn(len(lengths), hk, d, generator=g, device="cuda").to(torch.bfloat16)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = attend(q, kc, vc, table, n)
    for b in (*range(8), 700, 1369):
        one = attend(q[b:b + 1], kc, vc, table[b:b + 1], n[b:b + 1])
        assert torch.equal(out[b], one[0][0]) and torch.equal(lse[b], one[1][0]), b
    check((out[1:9], lse[1:9]), q[1:9], kc, vc, table[1:9], n[1:9])


def test_writes_count_as_changes_in_place():
    q, kc, vc, table, lengths = build([30, 5], 8, 2, 64, 16)
    k, v = torch.randn(2, 2, 2, 64, device="cuda").to(torch.bfloat16)
    seqs = torch.arange(2, device="cuda", dtype=torch.int32)
    before = [t._version for t in (kc, vc, q, k, v, lengths)]
    dc.kv_append(k, v, lengths - 1, seqs, table, kc, vc, q=q, q_out=q)
    assert [t._version - n for t, n in zip((kc, vc, q, k, v, lengths), before)] == [1, 1, 1, 0, 0, 0]
    out, lse, ws = torch.empty_like(q), torch.empty(2, 8, device="cuda"), dc.attention_workspace(2, 8, 2, 64, 32)
    dc.paged_attention(q, kc, vc, table, lengths, out, ws, lse=lse)
    assert (out._version, lse._version, kc._version - before[0]) == (1, 1, 1)


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (8, 2, 128), (6, 2, 192), (9, 1, 64), (12, 1, 96), (20, 1, 128), (64, 4, 128), (11, 1, 192),
                                     (48, 3, 256)])
def test_bits_of_binary16_do_not_depend_on_the_grid(hq, hk, d):
    """Low parts of the weights in rows of their own, in the same product or in a second one: the same sums."""
    q, kc, vc, table, lengths = build([1500, 33, 5, 260, 9000], hq, hk, d, 16, "f16")
    kc[2, 3, 0, :5] = 40.0
    vc[1, 2, 0, :7] = float("inf")
    kc[5, 1, 0] = 0.0
    q *= 4  # weights over the whole range
    want = attend(q, kc, vc, table, lengths)
    many = attend(q.repeat(60, 1, 1), kc, vc, table.repeat(60, 1), lengths.repeat(60))
    for i in (0, 59):
        for k in (0, 1):
            bits = torch.int16 if k == 0 else torch.int32
            assert torch.equal(many[k][5 * i:5 * i + 5].view(bits), want[k].view(bits))
    for b in range(5):
        one = attend(q[b:b + 1], kc, vc, table[b:b + 1], lengths[b:b + 1])
        assert torch.equal(one[0][0].view(torch.int16), want[0][b].view(torch.int16)) and torch.equal(one[1][0], want[1][b]), b
