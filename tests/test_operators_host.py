"""C-ABI checks of the language-model operators that need no GPU: bad argument
blocks are refused with a status before any CUDA call, good ones reach the
launch (which the ``test_fail_launch`` option reports as failed instead of
making it).  Pointers are fake device addresses.
"""
from __future__ import annotations

import math
import os
import shutil
import subprocess

import pytest

import reduce_copy_rank_gb300 as dc
from reduce_copy_rank_gb300 import _build, operators

OK, INVALID, ALIGN, OVERLAP, CUDA = 0, 1, 2, 3, 5
BASE = 0x7F00_0000_0000
MB = 1 << 20


def at(i: int) -> int:
    return BASE + i * 4096 * MB


@pytest.fixture(scope="module", autouse=True)
def built_library():
    _build.build()
    dc.lib()
    yield


@pytest.fixture(autouse=True)
def no_launch():
    with dc.options(test_fail_launch=1):
        yield


def score(**kw):
    f = dict(shards=[at(0), at(1)], widths=[500, 600], row_strides=[500, 640], tokens=at(2), logprobs=at(3), entropy=at(4),
             lse=at(5), top_logprobs=at(6), top_tokens=at(7), rows=9, vocab=1100, temperature=1.0, ranks=2, dtype=0,
             tokens_64=1, top_tokens_64=1, top=5)
    f.update(kw)
    return dc.dc_token_logprobs(**f)


def grad(**kw):
    f = dict(shards=[at(0), at(1)], widths=[500, 600], row_strides=[500, 640], grads=[at(2), at(3)],
             grad_row_strides=[500, 600], tokens=at(4), lse=at(5), entropy=at(6), grad_logprobs=at(7), grad_entropy=at(8),
             rows=9, vocab=1100, temperature=1.0, ranks=2, dtype=0, tokens_64=1)
    f.update(kw)
    return dc.dc_token_logprobs_backward(**f)


def append(**kw):
    f = dict(q=at(0), k=at(1), v=at(2), q_out=at(3), positions=at(4), seqs=at(5), page_table=at(6), cos_sin=at(7),
             k_cache=at(8), k_page_stride=16 * 2 * 64, k_slot_stride=2 * 64, k_cache_head_stride=64,
             v_cache=at(9), v_page_stride=16 * 2 * 64, v_slot_stride=2 * 64, v_cache_head_stride=64,
             q_token_stride=512, q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
             v_head_stride=64, q_out_token_stride=512, q_out_head_stride=64, tokens=7, table_rows=3, table_width=10,
             table_stride=10, cos_sin_rows=160, num_pages=30, page_size=16, q_heads=8, kv_heads=2, dim=64, rotary_dim=64)
    f.update(kw)
    return dc.dc_kv_append(**f)


def attend(**kw):
    f = dict(q=at(0), out=at(1), lse=at(2), page_table=at(3), lengths=at(4), workspace=at(5), workspace_bytes=64 * MB,
             k_cache=at(6), k_page_stride=16 * 2 * 64, k_slot_stride=2 * 64, k_cache_head_stride=64,
             v_cache=at(7), v_page_stride=16 * 2 * 64, v_slot_stride=2 * 64, v_cache_head_stride=64,
             q_seq_stride=512, q_head_stride=64, out_seq_stride=512, out_head_stride=64, seqs=3, table_width=100,
             table_stride=100, num_pages=30, page_size=16, q_heads=8, kv_heads=2, dim=64, scale=0.125)
    f.update(kw)
    return dc.dc_paged_attention(**f)


CALLS = [score, grad, append, attend]


@pytest.mark.parametrize("call", CALLS)
def test_good_arguments_reach_the_launch(call):
    before = dc.launch_count()
    assert call() == CUDA and "injected" in dc.last_error()
    assert dc.launch_count() == before


def test_null_blocks():
    L = operators._lib()
    for f in ("dc_token_logprobs", "dc_token_logprobs_backward", "dc_kv_append", "dc_paged_attention"):
        assert getattr(L, f)(None, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(ranks=0), INVALID), (dict(ranks=65), INVALID), (dict(rows=-1), INVALID), (dict(vocab=0), INVALID),
    (dict(vocab=1101), INVALID), (dict(vocab=(1 << 22) + 1), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
    (dict(temperature=0.0), INVALID), (dict(temperature=-1.0), INVALID), (dict(temperature=math.inf), INVALID),
    (dict(temperature=math.nan), INVALID), (dict(temperature=1e-60), INVALID), (dict(shards=0), INVALID),
    (dict(shards=[at(0), 0]), INVALID), (dict(shards=[at(0) + 1, at(1)]), ALIGN),
    (dict(shards=[at(0) + 2, at(1)], dtype=2), ALIGN), (dict(row_strides=[499, 640]), INVALID),
    (dict(row_strides=[1 << 62, 640]), INVALID), (dict(tokens=0), INVALID), (dict(tokens=at(2) + 4), ALIGN)])
def test_logits_checks(kw, want):
    assert score(**kw) == want, dc.last_error()
    if "top" not in kw:
        assert grad(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(top=-1), INVALID), (dict(top=33), INVALID), (dict(top=4, vocab=3), INVALID),
    (dict(top_logprobs=0, top_tokens=0), INVALID), (dict(logprobs=0), INVALID), (dict(logprobs=at(3) + 2), ALIGN),
    (dict(lse=at(3)), OVERLAP), (dict(lse=at(3) + 32), OVERLAP), (dict(entropy=at(0) + 1000), OVERLAP),
    (dict(logprobs=at(2)), OVERLAP), (dict(top_tokens=at(7) + 4), ALIGN),
    (dict(rows=0), OK), (dict(rows=0, logprobs=0, tokens=0), OK),
    (dict(entropy=0, lse=0, top=0, top_logprobs=0, top_tokens=0), CUDA), (dict(top_logprobs=0), CUDA),
    (dict(tokens=at(2) + 4, tokens_64=0), CUDA), (dict(shards=[at(0), 0], widths=[1100, 0], row_strides=[1100, 0]), CUDA),
    (dict(shards=[at(0), at(0) + 1000], row_strides=[1100, 1100]), CUDA)])
def test_score_checks(kw, want):
    assert score(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(grad_logprobs=0, grad_entropy=0), INVALID), (dict(entropy=0), INVALID), (dict(entropy=0, grad_entropy=0), CUDA),
    (dict(grad_logprobs=0), CUDA), (dict(lse=0), INVALID), (dict(grads=[at(2), 0]), INVALID),
    (dict(grads=[at(2), at(2)]), OVERLAP), (dict(grads=[at(0), at(3)]), CUDA),           # in place
    (dict(grads=[at(0), at(3)], grad_row_strides=[520, 600]), OVERLAP), (dict(grads=[at(0) + 2, at(3)]), OVERLAP),
    (dict(grads=[at(1), at(3)]), OVERLAP), (dict(grads=[at(5), at(3)]), OVERLAP),
    # columns of one tensor: apart, touching, and one column too many
    (dict(grads=[at(2), at(2) + 1000], grad_row_strides=[1100, 1100]), CUDA),
    (dict(grads=[at(2), at(2) + 998], grad_row_strides=[1100, 1100]), OVERLAP),
    (dict(grads=[at(2) + 1200, at(2)], grad_row_strides=[1100, 1100]), CUDA),
    (dict(grads=[at(2) + 1198, at(2)], grad_row_strides=[1100, 1100]), OVERLAP),
    (dict(grads=[at(2), at(2) + 1000], grad_row_strides=[1099, 1099]), OVERLAP),
    (dict(rows=0), OK)])
def test_grad_checks(kw, want):
    assert grad(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), INVALID), (dict(dim=60), INVALID), (dict(dim=1032), INVALID), (dict(dim=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(q_heads=-1), INVALID), (dict(rotary_dim=24), INVALID),
    (dict(rotary_dim=24, interleaved=1), CUDA), (dict(rotary_dim=20, interleaved=1), INVALID),
    (dict(rotary_dim=80), INVALID), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=0, cos_sin=0), CUDA),
    (dict(cos_sin=0), INVALID), (dict(cos_sin_rows=0), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=0), OK),
    (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(table_rows=0), INVALID),
    (dict(table_width=0), INVALID), (dict(table_stride=9), INVALID), (dict(k=at(1) + 8), ALIGN),
    (dict(k_token_stride=132), ALIGN), (dict(k_slot_stride=130), ALIGN), (dict(v=0), INVALID), (dict(q_out=0), INVALID),
    (dict(positions=at(4) + 2), ALIGN), (dict(v_cache=at(8)), OVERLAP), (dict(v_cache=at(8) + 256), CUDA),
    (dict(q_out=at(0)), CUDA), (dict(q_out=at(0), q_out_token_stride=1024), OVERLAP), (dict(q_out=at(1)), OVERLAP),
    (dict(k=at(8)), OVERLAP), (dict(q_out=at(9)), OVERLAP), (dict(page_table=at(8)), OVERLAP),
    (dict(q_heads=0, q=0, q_out=0), CUDA), (dict(k_page_stride=1 << 62), INVALID),
    # written tensors that fold onto themselves: a broadcast dimension, pages or heads that overlap
    (dict(q_out_token_stride=0), OVERLAP), (dict(q_out_head_stride=32), OVERLAP), (dict(k_page_stride=0), OVERLAP),
    (dict(v_slot_stride=64), OVERLAP), (dict(k_page_stride=16 * 2 * 64 - 8), OVERLAP),
    # heads outside tokens, and keys beside values
    (dict(k_slot_stride=64, k_cache_head_stride=16 * 64), CUDA), (dict(q_out_token_stride=64, q_out_head_stride=7 * 64), CUDA),
    (dict(k_page_stride=2 * 16 * 2 * 64, v_page_stride=2 * 16 * 2 * 64, v_cache=at(8) + 16 * 2 * 64 * 2), CUDA)])
def test_append_checks(kw, want):
    assert append(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(dim=80), INVALID), (dict(q_heads=7), INVALID), (dict(q_heads=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(window=-1), INVALID), (dict(scale=math.nan), INVALID), (dict(page_size=0), INVALID),
    (dict(seqs=-1), INVALID), (dict(seqs=0), OK), (dict(table_width=0), INVALID), (dict(table_stride=99), INVALID),
    (dict(num_pages=0), INVALID), (dict(workspace=0), INVALID), (dict(workspace=at(5) + 8), ALIGN),
    (dict(workspace_bytes=1024), INVALID), (dict(workspace_bytes=1024, table_width=8), CUDA),  # never split: not needed
    (dict(workspace_bytes=1024, window=128), CUDA), (dict(workspace=0, table_width=8), CUDA),
    (dict(q=at(0) + 8), ALIGN), (dict(q_head_stride=68), ALIGN), (dict(out=at(0)), OVERLAP), (dict(lse=at(1)), OVERLAP),
    (dict(workspace=at(6)), OVERLAP), (dict(out=at(7)), OVERLAP), (dict(lse=0), CUDA),
    (dict(table_width=1 << 30, page_size=16), INVALID), (dict(seqs=1, table_width=1 << 28, window=1000), CUDA),
    (dict(seqs=0x7FFFFFFF), INVALID), (dict(out_seq_stride=0), OVERLAP), (dict(out_head_stride=0), OVERLAP),
    (dict(k_page_stride=0), CUDA), (dict(q_seq_stride=0), CUDA)])  # what is only read may be broadcast
def test_attend_checks(kw, want):
    assert attend(**kw) == want, dc.last_error()


@pytest.mark.parametrize("seqs,hq,hk,dim,tokens", [
    (1, 8, 1, 128, 1000), (64, 32, 8, 128, 8192), (3, 64, 1, 256, 131072), (1, 1, 1, 64, 300), (1000, 12, 12, 64, 5000)])
def test_workspace_size_is_what_the_call_accepts(seqs, hq, hk, dim, tokens):
    n = dc.dc_attention_workspace_bytes(seqs, hq, hk, dim, tokens)
    call = dict(seqs=seqs, q_heads=hq, kv_heads=hk, dim=dim, table_width=tokens, table_stride=tokens, page_size=1,
                q_seq_stride=hq * dim, q_head_stride=dim, out_seq_stride=hq * dim, out_head_stride=dim,
                k_page_stride=hk * dim, k_slot_stride=hk * dim, k_cache_head_stride=dim, v_page_stride=hk * dim,
                v_slot_stride=hk * dim, v_cache_head_stride=dim)
    assert attend(workspace_bytes=n, **call) == CUDA, dc.last_error()
    assert attend(workspace_bytes=n - n // 20 - 1024, **call) == INVALID
    assert dc.dc_attention_workspace_bytes(seqs, hq, hk, dim, tokens // 2) <= n


def test_workspace_size_refusals():
    for a in ((1, 8, 3, 128, 100), (1, 8, 2, 100, 100), (-1, 8, 2, 128, 100), (1, 8, 2, 128, -1), (1, 8, 2, 128, 1 << 40)):
        assert dc.dc_attention_workspace_bytes(*a) == 0


def test_python_layouts_match_the_header(tmp_path):
    """The argument blocks that the binding packs have the size of the C structures."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "dc.h"\nint main(void){printf("%zu %zu %zu %zu\\n",'
                   "sizeof(dc_token_logprobs_t),sizeof(dc_token_logprobs_backward_t),sizeof(dc_kv_append_t),"
                   "sizeof(dc_paged_attention_t));return 0;}\n")
    exe = tmp_path / "sizes"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    blocks = (operators._SCORE, operators._GRAD, operators._APPEND, operators._ATTEND)
    assert sizes == [len(b.of({})) for b in blocks]


def test_unknown_fields_are_refused():
    with pytest.raises(TypeError):
        dc.dc_token_logprobs(shard=[1])


@pytest.mark.parametrize("temperature,want", [
    (1e-38, CUDA), (4.3e-39, CUDA), (4.2e-39, INVALID), (3e-39, INVALID), (1e30, CUDA), (1.1e30, INVALID)])
def test_temperatures_whose_exponents_do_not_fit_binary32(temperature, want):
    """log2(e) / temperature is at most FLT_MAX (3.4028e38, from 4.2397e-39 on), 1 / temperature at least 1e-30."""
    assert score(temperature=temperature) == want, dc.last_error()
    assert grad(temperature=temperature) == want, dc.last_error()


# queries, keys and values as heads of one tensor of 12 heads of 64 a token, the queries rotated in place
FUSED = dict(q_out=at(0), k=at(0) + 8 * 128, v=at(0) + 10 * 128, q_token_stride=768, q_out_token_stride=768, k_token_stride=768,
             v_token_stride=768)
# ... and of 2 heads of each, side by side head by head
TURNS = dict(q_out=at(0), k=at(0) + 128, v=at(0) + 256, q_heads=2, **{f"{x}_token_stride": 384 for x in ("q", "k", "v", "q_out")},
             **{f"{x}_head_stride": 192 for x in ("q", "k", "v", "q_out")})


@pytest.mark.parametrize("kw,want", [
    ({}, CUDA), (dict(q=at(0) + 512, q_out=at(0) + 512, k=at(0), v=at(0) + 256), CUDA), (dict(k=at(1), v=at(2)), CUDA),
    (dict(tokens=1), CUDA), (dict(tokens=1, k=at(0) + 7 * 128), OVERLAP),
    (dict(k=at(0)), OVERLAP), (dict(v=at(0)), OVERLAP),                            # keys or values are queries
    (dict(k=at(0) + 7 * 128), OVERLAP), (dict(v=at(0) + 128), OVERLAP),            # share a head, or are one head on
    (dict(k=at(0) + 8 * 128 - 16), OVERLAP), (dict(v=at(0) + 11 * 128), OVERLAP),  # end or begin inside one; the next token's
    (dict(k=at(0) + 768 * 2), OVERLAP), (dict(v=at(0) + 3 * 768 * 2 + 5 * 128), OVERLAP),  # a later token's queries
    (dict(k_token_stride=0), CUDA), (dict(k=at(0) + 128, k_token_stride=0), OVERLAP),  # one token's keys for all
    (dict(k_head_stride=0), CUDA), (dict(k=at(0) + 7 * 128, k_head_stride=0), OVERLAP),
    (dict(k_token_stride=1536), CUDA), (dict(k=at(0) + 6 * 128, k_token_stride=1536), OVERLAP),
    (dict(k_token_stride=776), OVERLAP),                                           # cannot be shown apart (and is not)
    (dict(TURNS), CUDA), (dict(TURNS, k=at(0)), OVERLAP), (dict(TURNS, v=at(0) + 384), OVERLAP),
    (dict(TURNS, k=at(0) + 112), OVERLAP), (dict(TURNS, k=at(0) + 144, v=at(0) + 256), CUDA),
    # heads outside tokens: 7 tokens of 64 a head
    (dict(k=at(0) + 8 * 7 * 128, v=at(0) + 10 * 7 * 128, **{f"{x}_token_stride": 64 for x in ("q", "k", "v", "q_out")},
          **{f"{x}_head_stride": 448 for x in ("q", "k", "v", "q_out")}), CUDA),
    (dict(k=at(0) + 7 * 7 * 128, v=at(0) + 10 * 7 * 128, **{f"{x}_token_stride": 64 for x in ("q", "k", "v", "q_out")},
          **{f"{x}_head_stride": 448 for x in ("q", "k", "v", "q_out")}), OVERLAP)])
def test_queries_in_place_share_nothing_with_keys_and_values(kw, want):
    assert append(**{**FUSED, **kw}) == want, dc.last_error()


def test_overlap_of_queries_in_place_against_every_byte():
    """Random layouts: whatever shares a byte is refused, and what shares none in one fused layout is not."""
    import random

    rng = random.Random(11)
    seen = {CUDA: 0, OVERLAP: 0}
    for _ in range(4000):
        n, hq, hk, unit = rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 2), 8 * rng.choice([1, 2, 4])
        dim = 8 * rng.randint(1, 3)

        def strides(heads):
            head = unit * rng.randint(1, 4) if rng.random() < 0.8 else 0
            token = unit * rng.randint(1, 14)
            return token, head

        qt, qh = strides(hq)
        kt, kh = strides(hk) if rng.random() < 0.4 else (qt, qh)
        base = at(0) + 4096
        k = base + 2 * unit * rng.randint(-8, 24)

        def covered(p, heads, t, h):
            return {p + 2 * (i * t + j * h + e) for i in range(n) for j in range(heads) for e in range(dim)}

        got = append(q=base, q_out=base, k=k, tokens=n, q_heads=hq, kv_heads=hk, dim=dim, rotary_dim=0, cos_sin=0,
                     q_token_stride=qt, q_head_stride=qh, q_out_token_stride=qt, q_out_head_stride=qh, k_token_stride=kt,
                     k_head_stride=kh, k_page_stride=16 * hk * 64, v_page_stride=16 * hk * 64, k_slot_stride=hk * 64,
                     v_slot_stride=hk * 64)
        if got == OVERLAP and "q_out: its rows" in dc.last_error():
            continue
        shared = covered(base, hq, qt, qh) & covered(k, hk, kt, kh)
        assert got in (CUDA, OVERLAP), dc.last_error()
        assert got == OVERLAP or not shared, (n, hq, hk, dim, qt, qh, kt, kh, k - base)
        seen[got] += 1
    assert min(seen.values()) > 500, seen


# both caches in one tensor: strides of a token's 2 heads of 64, of a page of 16 tokens
def both(page, slot, head, v, **kw):
    return dict(k_page_stride=page, v_page_stride=page, k_slot_stride=slot, v_slot_stride=slot, k_cache_head_stride=head,
                v_cache_head_stride=head, v_cache=at(8) + 2 * v, **kw)


@pytest.mark.parametrize("kw,want", [
    (both(4096, 128, 64, 2048), CUDA), (both(2048, 128, 64, 2048 * 30), CUDA),         # page by page; one after the other
    (both(4096, 256, 64, 128), CUDA), (both(4096, 256, 128, 64), CUDA),                # token by token, head by head
    (both(4096, 64, 2048, 1024), CUDA), (both(4096, 128, 1024 * 2, 64), CUDA),         # the same with heads outside tokens
    (both(2048, 128, 64, 0, num_pages=1), OVERLAP), (both(2048, 128, 64, 2048, num_pages=1), CUDA),
    (both(2048, 128, 64, 128), OVERLAP), (both(2048, 128, 64, 64), OVERLAP), (both(2048, 128, 64, 8), OVERLAP),
    (both(2048, 128, 64, 2048), OVERLAP), (both(2048, 128, 64, 2048 * 29 + 1920), OVERLAP),  # one page on; the last slot
    (both(4096, 128, 64, 1984), OVERLAP), (both(4096, 128, 64, 2112), OVERLAP),        # a head into the other's page
    (both(4096, 256, 64, 192), OVERLAP), (both(4096, 256, 128, 72), OVERLAP), (both(4096, 64, 2048, 960), OVERLAP),
    (dict(both(4096, 128, 64, 2048), v_slot_stride=64, v_cache_head_stride=1024), CUDA),  # laid out differently inside pages
    (dict(both(4096, 128, 64, 2048), v_page_stride=8192), CUDA), (dict(both(4096, 128, 64, 2048), v_page_stride=6144), OVERLAP),
    (dict(both(4096, 128, 64, 2048), k_cache=at(8) + 4096, v_cache=at(8)), CUDA)])
def test_caches_share_nothing(kw, want):
    assert append(**kw) == want, dc.last_error()


def test_python_layouts_have_the_headers_offsets(tmp_path):
    """Every field of the argument blocks lies where the C structures have it."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    caches = {f"{x}{a}": f"{x}_cache.{b}" for x in "kv" for a, b in (
        ("_cache", "data"), ("_page_stride", "page_stride"), ("_slot_stride", "token_stride"), ("_cache_head_stride", "head_stride"))}
    blocks = {"dc_token_logprobs_t": operators._SCORE, "dc_token_logprobs_backward_t": operators._GRAD,
              "dc_kv_append_t": operators._APPEND, "dc_paged_attention_t": operators._ATTEND}
    lines = [f'printf("%zu\\n", offsetof({t}, {caches.get(n, n)}));' for t, b in blocks.items() for n in b.names]
    src = tmp_path / "offsets.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dc.h"\nint main(void){' + "\n".join(lines) + "return 0;}\n")
    exe = tmp_path / "offsets"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    want = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    # a field whose lowest byte alone is not 0 (little-endian: the number's first byte)
    least = {"temperature": 2.0 ** -1074, "scale": 2.0 ** -149}
    got = [b.of({n: least.get(n, 1)}).index(1) for b in blocks.values() for n in b.names]
    assert got == want
