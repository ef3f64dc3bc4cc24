"""C-ABI checks of the operators around a rollout and a training step on it that
need no GPU: bad argument blocks are refused with a status before any CUDA call,
good ones reach the launch (which the ``test_fail_launch`` option reports as
failed instead of making it).  Pointers are fake device addresses.
"""
from __future__ import annotations

import math
import os
import random
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


def linear(**kw):
    f = dict(hidden=at(0), weights=[at(1), at(2)], widths=[500, 600], weight_row_strides=[64, 72], tokens=at(3), logprobs=at(4),
             entropy=at(5), lse=at(6), workspace=at(7), workspace_bytes=64 * MB, hidden_row_stride=64, rows=9, hidden_size=64,
             vocab=1100, temperature=1.0, ranks=2, dtype=0, tokens_64=1)
    f.update(kw)
    return dc.dc_linear_logprobs(**f)


def linear_grad(**kw):
    f = dict(hidden=at(0), weights=[at(1), at(2)], widths=[500, 600], weight_row_strides=[64, 72], tokens=at(3), lse=at(4),
             entropy=at(5), grad_logprobs=at(6), grad_entropy=at(7), grad_hidden=at(8), grad_weights=[at(9), at(10)],
             grad_weight_row_strides=[64, 64], workspace=at(11), workspace_bytes=64 * MB, hidden_row_stride=64,
             grad_hidden_row_stride=64, rows=9, hidden_size=64, vocab=1100, temperature=1.0, ranks=2, dtype=0, tokens_64=1)
    f.update(kw)
    return dc.dc_linear_logprobs_backward(**f)


def append_norm(**kw):
    f = dict(q=at(0), k=at(1), v=at(2), q_out=at(3), positions=at(4), seqs=at(5), page_table=at(6), cos_sin=at(7),
             k_cache=at(8), k_page_stride=16 * 2 * 64, k_slot_stride=2 * 64, k_cache_head_stride=64,
             v_cache=at(9), v_page_stride=16 * 2 * 64, v_slot_stride=2 * 64, v_cache_head_stride=64,
             q_token_stride=512, q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
             v_head_stride=64, q_out_token_stride=512, q_out_head_stride=64, tokens=7, table_rows=3, table_width=10,
             table_stride=10, cos_sin_rows=160, num_pages=30, page_size=16, q_heads=8, kv_heads=2, dim=64, rotary_dim=64,
             q_norm=at(10), k_norm=at(11), eps=1e-6)
    f.update(kw)
    return dc.dc_kv_append_norm(**f)


def heads(**where):
    """Tensors of 8 query or 2 key heads of 64, one after the other or as given."""
    f = {}
    for name, (base, hk) in where.items():
        f |= {name: base, f"{name}_token_stride": hk * 64, f"{name}_head_stride": 64}
    return f


def norm(**kw):
    f = heads(q=(at(0), 8), k=(at(1), 2), q_out=(at(2), 8), k_out=(at(3), 2)) | dict(
        positions=at(4), cos_sin=at(5), q_norm=at(6), k_norm=at(7), tokens=7, cos_sin_rows=160, q_heads=8, kv_heads=2, dim=64,
        rotary_dim=64, eps=1e-6)
    f.update(kw)
    return dc.dc_qk_norm_rotate(**f)


def norm_grad(**kw):
    f = heads(q=(at(0), 8), k=(at(1), 2), grad_q_out=(at(2), 8), grad_k_out=(at(3), 2), grad_q=(at(4), 8), grad_k=(at(5), 2)) | dict(
        positions=at(6), cos_sin=at(7), q_norm=at(8), k_norm=at(9), grad_q_norm=at(10), grad_k_norm=at(11), workspace=at(12),
        workspace_bytes=MB, tokens=7, cos_sin_rows=160, q_heads=8, kv_heads=2, dim=64, rotary_dim=64, eps=1e-6)
    f.update(kw)
    return dc.dc_qk_norm_rotate_backward(**f)


def prefix(**kw):
    f = dict(q=at(0), out=at(1), lse=at(2), page_table=at(3), lengths=at(4), workspace=at(5), workspace_bytes=256 * MB,
             k_cache=at(6), k_page_stride=16 * 2 * 64, k_slot_stride=2 * 64, k_cache_head_stride=64,
             v_cache=at(7), v_page_stride=16 * 2 * 64, v_slot_stride=2 * 64, v_cache_head_stride=64,
             q_seq_stride=512, q_head_stride=64, out_seq_stride=512, out_head_stride=64, seqs=6, table_width=100,
             table_stride=100, num_pages=30, page_size=16, q_heads=8, kv_heads=2, dim=64, scale=0.125,
             prefix_table=at(8), prefix_lengths=at(9), prefixes=2, prefix_table_width=50, prefix_table_stride=50)
    f.update(kw)
    return dc.dc_prefix_attention(**f)


CALLS = [linear, linear_grad, append_norm, norm, norm_grad, prefix]


@pytest.mark.parametrize("call", CALLS)
def test_good_arguments_reach_the_launch(call):
    before = dc.launch_count()
    assert call() == CUDA and "injected" in dc.last_error()
    assert dc.launch_count() == before


def test_null_blocks():
    L = operators._lib()
    for f in operators._ENTRIES:
        assert getattr(L, f)(None, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(ranks=0), INVALID), (dict(ranks=65), INVALID), (dict(rows=-1), INVALID), (dict(rows=(1 << 24) + 1), INVALID),
    (dict(vocab=0), INVALID), (dict(vocab=1101), INVALID), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(hidden_size=0), INVALID), (dict(hidden_size=60), INVALID), (dict(hidden_size=(1 << 20) + 8), INVALID),
    (dict(temperature=0.0), INVALID), (dict(temperature=math.nan), INVALID), (dict(temperature=1e-60), INVALID),
    (dict(weights=0), INVALID), (dict(weights=[at(1), 0]), INVALID), (dict(weights=[at(1) + 8, at(2)]), ALIGN),
    (dict(hidden=0), INVALID), (dict(hidden=at(0) + 8), ALIGN), (dict(hidden_row_stride=68), ALIGN),
    (dict(hidden_row_stride=56), INVALID), (dict(weight_row_strides=[60, 72]), INVALID), (dict(weight_row_strides=[68, 72]), ALIGN),
    (dict(weight_row_strides=[1 << 40, 72]), INVALID), (dict(tokens=0), INVALID), (dict(tokens=at(3) + 4), ALIGN),
    (dict(tokens=at(3) + 4, tokens_64=0), CUDA), (dict(workspace=0), INVALID), (dict(workspace=at(7) + 128), ALIGN),
    (dict(workspace_bytes=1000), INVALID), (dict(weights=[at(1), 0], widths=[1100, 0]), CUDA),
    (dict(hidden_row_stride=0, rows=1), CUDA), (dict(widths=[500, 5_000_000]), INVALID)])
def test_head_checks(kw, want):
    assert linear(**kw) == want, dc.last_error()
    if "workspace" in kw:
        kw = {k: v + (4 * 4096 * MB if k == "workspace" and v else 0) for k, v in kw.items()}
    assert linear_grad(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(logprobs=0), INVALID), (dict(logprobs=at(4) + 2), ALIGN), (dict(entropy=0, lse=0), CUDA), (dict(lse=at(4)), OVERLAP),
    (dict(lse=at(4) + 32), OVERLAP), (dict(entropy=at(0) + 100), OVERLAP), (dict(logprobs=at(3)), OVERLAP),
    (dict(workspace=at(1)), OVERLAP), (dict(workspace=at(4)), OVERLAP), (dict(entropy=at(2) + 64), OVERLAP),
    (dict(rows=0), OK), (dict(rows=0, hidden=0, tokens=0, logprobs=0, workspace=0), OK)])
def test_linear_checks(kw, want):
    assert linear(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(grad_logprobs=0, grad_entropy=0), INVALID), (dict(entropy=0), INVALID), (dict(entropy=0, grad_entropy=0), CUDA),
    (dict(grad_logprobs=0), CUDA), (dict(lse=0), INVALID), (dict(grad_hidden=0), CUDA), (dict(grad_weights=0), CUDA),
    (dict(grad_hidden=0, grad_weights=0), INVALID), (dict(grad_weights=[at(9), 0]), INVALID),
    (dict(grad_weights=[at(9), at(10) + 8]), ALIGN), (dict(grad_weight_row_strides=[64, 60]), INVALID),
    (dict(grad_weight_row_strides=0), INVALID), (dict(grad_hidden=at(8) + 8), ALIGN), (dict(grad_hidden_row_stride=68), ALIGN),
    # outputs meet neither one another nor what is read, not even exactly
    (dict(grad_hidden=at(0)), OVERLAP), (dict(grad_hidden=at(1)), OVERLAP), (dict(grad_weights=[at(1), at(10)]), OVERLAP),
    (dict(grad_weights=[at(9), at(9) + 499 * 128]), OVERLAP), (dict(grad_weights=[at(9), at(9) + 500 * 128]), CUDA),
    (dict(grad_weights=[at(9), at(0)]), OVERLAP), (dict(grad_hidden=at(9) + 1280), OVERLAP), (dict(grad_hidden=at(6)), OVERLAP),
    (dict(grad_weights=[at(3), at(10)]), OVERLAP), (dict(workspace=at(8)), OVERLAP), (dict(workspace=at(10)), OVERLAP),
    (dict(workspace=at(4)), OVERLAP),
    # rows of the gradient of one shard beside those of the other
    (dict(grad_weights=[at(9), at(9) + 128], grad_weight_row_strides=[128, 128]), CUDA),
    (dict(grad_weights=[at(9), at(9) + 112], grad_weight_row_strides=[128, 128]), OVERLAP),
    (dict(rows=0, grad_weights=0), OK), (dict(rows=0), CUDA)])
def test_linear_grad_checks(kw, want):
    assert linear_grad(**kw) == want, dc.last_error()


@pytest.mark.parametrize("rows,size,widths,vocab", [
    (1, 8, [1], 1), (300, 1000, [1000, 1, 513], 1514), (4096, 4096, [16000] * 8, 127900), (7, 64, [3] * 64, 192),
    (128, 512, [40000, 24577], 64577), (33, 8192, [200000], 200000)])
def test_workspace_sizes_are_what_the_calls_accept(rows, size, widths, vocab):
    call = dict(rows=rows, hidden_size=size, vocab=vocab, widths=widths, ranks=len(widths), hidden_row_stride=size,
                weights=[at(40 + i) for i in range(len(widths))], weight_row_strides=[size] * len(widths))
    n = dc.dc_linear_logprobs_workspace_bytes(rows, size, sum(widths), False)
    assert linear(workspace_bytes=n, **call) == CUDA, dc.last_error()
    assert linear(workspace_bytes=rows * sum(-(-w // 256) for w in widths) * 16, **call) == INVALID
    n = dc.dc_linear_logprobs_workspace_bytes(rows, size, sum(widths), True)
    call |= dict(grad_weights=[at(140 + i) for i in range(len(widths))], grad_weight_row_strides=[size] * len(widths),
                 grad_hidden_row_stride=size)
    assert linear_grad(workspace_bytes=n, **call) == CUDA, dc.last_error()
    assert linear_grad(workspace_bytes=rows * min(max(widths), 16384) * 2, **call) == INVALID
    # (kept from vocabulary to vocabulary: the gradient's does not grow with it)
    assert n <= 256 + rows * (24576 * 2 + max(4096 + 256 * 16, size) * 4) + 1024


def test_workspace_size_refusals():
    for a in ((-1, 64, 100), (3, 60, 100), (3, 0, 100), (3, 64, 0), (3, 64, (1 << 22) + 1), ((1 << 24) + 1, 64, 100)):
        assert dc.dc_linear_logprobs_workspace_bytes(*a, False) == 0
    for a in ((-1, 8, 2, 64), (3, 0, 2, 64), (3, 8, 0, 64), (3, 8, 2, 520), (3, 8, 2, 6)):
        assert dc.dc_qk_norm_workspace_bytes(*a) == 0
    for a in ((5, 2, 8, 2, 64, 100, 100), (4, 0, 8, 2, 64, 100, 100), (4, 2, 8, 3, 64, 100, 100), (4, 2, 8, 2, 80, 100, 100),
              (4, 2, 8, 2, 64, -1, 100), (4, 2, 8, 2, 64, 100, 1 << 40), (4, 2, 8, 2, 64, 1 << 40, 100)):
        assert dc.dc_prefix_attention_workspace_bytes(*a) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dim=520, rotary_dim=64), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(eps=0.0), CUDA), (dict(k_norm=0), INVALID), (dict(q_norm=0), INVALID), (dict(q_norm=0, q_heads=0, q=0, q_out=0), CUDA),
    (dict(k_norm=at(11) + 1), ALIGN), (dict(k_norm=at(11) + 2), CUDA), (dict(k_norm=at(11) + 2, norm_32=1), ALIGN),
    (dict(q_norm=at(3)), OVERLAP), (dict(k_norm=at(8) + 64), OVERLAP), (dict(k_norm=at(9)), OVERLAP), (dict(q_norm=at(11)), CUDA),
    # what kv_append refuses
    (dict(dim=60), INVALID), (dict(rotary_dim=24), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=0), OK), (dict(page_size=0), INVALID),
    (dict(q_out=at(1)), OVERLAP), (dict(v_cache=at(8)), OVERLAP), (dict(q_out=at(0)), CUDA), (dict(k=at(1) + 8), ALIGN),
    (dict(q_out_token_stride=0), OVERLAP), (dict(cos_sin=0), INVALID), (dict(rotary_dim=0, cos_sin=0), CUDA)])
def test_append_norm_checks(kw, want):
    assert append_norm(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), INVALID), (dict(dim=520, rotary_dim=64), INVALID), (dict(dim=60), INVALID), (dict(dim=0), INVALID),
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(rotary_dim=24), INVALID), (dict(rotary_dim=24, interleaved=1), CUDA),
    (dict(rotary_dim=80), INVALID), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=0, cos_sin=0), CUDA), (dict(cos_sin=0), INVALID),
    (dict(cos_sin_rows=0), INVALID), (dict(eps=-1e-6), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=0), OK),
    (dict(positions=0), INVALID), (dict(positions=at(4) + 2), ALIGN), (dict(q_norm=0), INVALID), (dict(k_norm=at(7) + 1), ALIGN),
    (dict(k_norm=at(7) + 2, norm_32=1), ALIGN), (dict(q=0), INVALID), (dict(q=at(0) + 8), ALIGN), (dict(k_token_stride=132), ALIGN)])
def test_norm_checks(kw, want):
    assert norm(**kw) == want, dc.last_error()
    moved = {"positions": 2, "q_norm": 2, "k_norm": 2}
    if not (set(kw) == {"tokens"} and want == OK):
        assert norm_grad(**{k: v + moved.get(k, 0) * 4096 * MB if v and k in moved else v for k, v in kw.items()}) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(q_out=at(0)), CUDA), (dict(k_out=at(1)), CUDA), (dict(q_out=at(0), k_out=at(1)), CUDA), (dict(q_out=at(1)), OVERLAP),
    (dict(q_out=at(0), q_out_token_stride=1024), OVERLAP), (dict(k_out=at(0)), OVERLAP), (dict(k_out=at(2)), OVERLAP),
    (dict(q_out=at(0) + 128), OVERLAP), (dict(q_out_token_stride=0), OVERLAP), (dict(q_out_head_stride=32), OVERLAP),
    (dict(q_out=at(4)), OVERLAP), (dict(k_out=at(5)), OVERLAP), (dict(k_out=at(6)), OVERLAP), (dict(q_out=0), INVALID),
    # queries and keys as heads of one tensor, and their results beside one another in another, or in place
    (dict(k=at(0) + 8 * 128, q_token_stride=640, k_token_stride=640), CUDA),
    (dict(k=at(0) + 8 * 128, q_token_stride=640, k_token_stride=640, q_out=at(0), k_out=at(0) + 8 * 128, q_out_token_stride=640,
          k_out_token_stride=640), CUDA),
    (dict(k=at(0) + 8 * 128, q_token_stride=640, k_token_stride=640, q_out=at(0), q_out_token_stride=640, k_out=at(0)), OVERLAP),
    (dict(k_out=at(2) + 8 * 128, q_out_token_stride=640, k_out_token_stride=640), CUDA),
    (dict(k_out=at(2) + 7 * 128, q_out_token_stride=640, k_out_token_stride=640), OVERLAP),
    (dict(q_token_stride=0), CUDA), (dict(k_head_stride=0), CUDA)])  # what is only read may be broadcast
def test_norm_overlaps(kw, want):
    assert norm(**kw) == want, dc.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(grad_q=at(2)), CUDA), (dict(grad_q=at(2), grad_k=at(3)), CUDA), (dict(grad_q=at(0)), OVERLAP), (dict(grad_k=at(1)), OVERLAP),
    (dict(grad_q=at(3)), OVERLAP), (dict(grad_k=at(4)), OVERLAP), (dict(grad_q_token_stride=0), OVERLAP),
    (dict(grad_q=at(2), grad_q_head_stride=128, grad_q_token_stride=1024), OVERLAP), (dict(grad_q=at(8)), OVERLAP),
    (dict(grad_q_norm=0), CUDA), (dict(grad_q_norm=0, grad_k_norm=0), CUDA), (dict(grad_q_norm=0, grad_k_norm=0, workspace=0, workspace_bytes=0), CUDA),
    (dict(workspace=0), INVALID), (dict(workspace_bytes=1000), INVALID), (dict(workspace=at(12) + 8), ALIGN),
    (dict(grad_q_norm=at(11)), OVERLAP), (dict(grad_q_norm=at(8)), OVERLAP), (dict(grad_k_norm=at(5)), OVERLAP),
    (dict(workspace=at(0)), OVERLAP), (dict(workspace=at(4)), OVERLAP), (dict(workspace=at(10)), OVERLAP), (dict(grad_k_norm=at(11) + 1), ALIGN),
    (dict(tokens=0, grad_q_norm=0, grad_k_norm=0), OK), (dict(tokens=0), CUDA), (dict(tokens=0, workspace=0, q=0, positions=0), CUDA)])
def test_norm_grad_checks(kw, want):
    assert norm_grad(**kw) == want, dc.last_error()


def test_heads_in_place_against_every_byte():
    """Random layouts: outputs that share a byte with what is read, or with each other, are refused."""
    rng = random.Random(5)
    seen = {CUDA: 0, OVERLAP: 0}
    for _ in range(4000):
        n, hq, hk, dim = rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 2), 8 * rng.randint(1, 3)
        base = at(0) + 4096
        layout = {}
        covered = {}
        same = rng.random() < 0.6
        token, head = 8 * rng.randint(1, 40), 8 * rng.randint(1, 6)
        for name, count in (("q", hq), ("k", hk), ("q_out", hq), ("k_out", hk)):
            t, h = (token, head) if same else (8 * rng.randint(1, 40), 8 * rng.randint(1, 6))
            p = base + 16 * rng.randint(0, 60)
            if name.endswith("_out") and rng.random() < 0.3:
                src = name[0]
                p, t, h = layout[src], layout[f"{src}_token_stride"], layout[f"{src}_head_stride"]
            layout |= {name: p, f"{name}_token_stride": t, f"{name}_head_stride": h}
            covered[name] = [p + 2 * (i * t + j * h + e) for i in range(n) for j in range(count) for e in range(dim)]
        got = norm(tokens=n, q_heads=hq, kv_heads=hk, dim=dim, rotary_dim=0, cos_sin=0, **layout)
        assert got in (CUDA, OVERLAP), dc.last_error()
        seen[got] += 1
        if got == OVERLAP:
            continue
        for out in ("q_out", "k_out"):
            assert len(set(covered[out])) == len(covered[out])
            for other in covered:
                exact = other == out[0] and all(layout[out + s] == layout[other + s] for s in ("", "_token_stride", "_head_stride"))
                if other != out and not exact:
                    assert not set(covered[out]) & set(covered[other]), (layout, out, other)
    assert min(seen.values()) > 100, seen


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(dim=80), INVALID), (dict(q_heads=7), INVALID), (dict(window=5), INVALID), (dict(scale=math.nan), INVALID),
    (dict(page_size=0), INVALID), (dict(seqs=-1), INVALID), (dict(seqs=0), OK), (dict(table_width=0), INVALID), (dict(prefixes=0), INVALID),
    (dict(prefixes=4), INVALID), (dict(prefixes=-1), INVALID), (dict(prefixes=6), CUDA), (dict(prefixes=1), CUDA),
    (dict(prefix_table_width=0), INVALID), (dict(prefix_table_width=-1), INVALID), (dict(prefix_table_stride=49), INVALID),
    (dict(prefix_table_stride=49, prefixes=1), CUDA), (dict(prefix_table=0), INVALID), (dict(prefix_lengths=0), INVALID),
    (dict(prefix_table=at(8) + 2), ALIGN), (dict(prefix_lengths=at(9) + 2), ALIGN), (dict(prefix_table_width=1 << 30, prefix_table_stride=1 << 30), INVALID),
    (dict(workspace=0), INVALID), (dict(workspace=at(5) + 8), ALIGN), (dict(workspace_bytes=MB), INVALID),
    (dict(workspace_bytes=MB, table_width=8), INVALID), (dict(workspace=0, table_width=8), INVALID),
    (dict(workspace=at(6)), OVERLAP), (dict(workspace=at(8)), OVERLAP), (dict(workspace=at(1)), OVERLAP), (dict(workspace=at(6), table_width=8), OVERLAP),
    (dict(workspace=at(9), table_width=8), OVERLAP), (dict(out=at(0)), OVERLAP), (dict(out=at(8)), OVERLAP), (dict(lse=at(9)), OVERLAP),
    (dict(lse=0), CUDA), (dict(q=at(0) + 8), ALIGN), (dict(out_seq_stride=0), OVERLAP), (dict(q_seq_stride=0), CUDA), (dict(k_page_stride=0), CUDA)])
def test_prefix_checks(kw, want):
    assert prefix(**kw) == want, dc.last_error()


@pytest.mark.parametrize("seqs,prefixes,hq,hk,dim,shared,own", [
    (1, 1, 8, 1, 128, 1000, 100), (64, 2, 32, 8, 128, 65536, 1024), (6, 3, 64, 1, 256, 131072, 1), (1, 1, 1, 1, 64, 1, 1),
    (1000, 1, 12, 12, 64, 5000, 5000)])
def test_prefix_workspace_size_is_what_the_call_accepts(seqs, prefixes, hq, hk, dim, shared, own):
    n = dc.dc_prefix_attention_workspace_bytes(seqs, prefixes, hq, hk, dim, shared, own)
    call = dict(seqs=seqs, prefixes=prefixes, q_heads=hq, kv_heads=hk, dim=dim, table_width=own, table_stride=own, page_size=1,
                prefix_table_width=shared, prefix_table_stride=shared, q_seq_stride=hq * dim, q_head_stride=dim,
                out_seq_stride=hq * dim, out_head_stride=dim, k_page_stride=hk * dim, k_slot_stride=hk * dim,
                k_cache_head_stride=dim, v_page_stride=hk * dim, v_slot_stride=hk * dim, v_cache_head_stride=dim)
    assert prefix(workspace_bytes=n, **call) == CUDA, dc.last_error()
    assert prefix(workspace_bytes=n - 1, **call) == INVALID
    assert dc.dc_prefix_attention_workspace_bytes(seqs, prefixes, hq, hk, dim, max(1, shared // 2), own) <= n


def blocks():
    return {"dc_linear_logprobs_t": operators._LINEAR, "dc_linear_logprobs_backward_t": operators._LINEAR_GRAD,
            "dc_kv_append_norm_t": operators._APPEND_NORM, "dc_qk_norm_rotate_t": operators._NORM,
            "dc_qk_norm_rotate_backward_t": operators._NORM_GRAD, "dc_prefix_attention_t": operators._PREFIX}


def test_python_layouts_have_the_headers_sizes_and_offsets(tmp_path):
    """The argument blocks that the binding packs have the C structures' sizes, and every field lies where they have it."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    caches = {f"{x}{a}": f"{x}_cache.{b}" for x in "kv" for a, b in (
        ("_cache", "data"), ("_page_stride", "page_stride"), ("_slot_stride", "token_stride"), ("_cache_head_stride", "head_stride"))}

    def member(struct, name):
        if struct in ("dc_kv_append_norm_t", "dc_prefix_attention_t"):
            inner, own = ("append", operators._APPEND) if "append" in struct else ("own", operators._ATTEND)
            if name in own.names:
                return f"{inner}.{caches.get(name, name)}"
            return name
        if "norm_rotate" in struct:
            for s in ("_token_stride", "_head_stride"):
                if name.endswith(s):
                    return f"{name[:-len(s)]}.{s[1:]}"
            if name in ("q", "k", "q_out", "k_out", "grad_q_out", "grad_k_out", "grad_q", "grad_k"):
                return f"{name}.data"
        return name

    lines = [f'printf("%zu\\n", sizeof({t}));' for t in blocks()]
    lines += [f'printf("%zu\\n", offsetof({t}, {member(t, n)}));' for t, b in blocks().items() for n in b.names]
    src = tmp_path / "offsets.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dc.h"\nint main(void){' + "\n".join(lines) + "return 0;}\n")
    exe = tmp_path / "offsets"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    want = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    # a field whose lowest byte alone is not 0 (little-endian: the number's first byte)
    least = {"temperature": 2.0 ** -1074, "scale": 2.0 ** -149, "eps": 2.0 ** -149}
    got = [len(b.of({})) for b in blocks().values()]
    got += [b.of({n: least.get(n, 1)}).index(1) for b in blocks().values() for n in b.names]
    assert got == want


def test_unknown_fields_are_refused():
    with pytest.raises(TypeError):
        dc.dc_linear_logprobs(weight=[1])
    with pytest.raises(TypeError):
        dc.dc_prefix_attention(prefix=1)


def test_tensors_off_the_gpu_and_of_wrong_shapes_are_refused():
    """The tensor functions' own checks, on CPU tensors: no CUDA call is made."""
    torch = pytest.importorskip("torch")
    b = torch.bfloat16
    x, w, t, f = torch.zeros(3, 16, dtype=b), [torch.zeros(20, 16, dtype=b)], torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="hidden must be a CUDA tensor"):
        dc.linear_logprobs(x, w, t, f, ws)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        dc.linear_logprobs(x.float(), w, t, f, ws)
    with pytest.raises(ValueError, match="expected .rows, hidden size."):
        dc.linear_logprobs(x[0], w, t, f, ws)
    with pytest.raises(TypeError, match="must be a tensor"):
        dc.linear_logprobs(None, w, t, f, ws)
    q, k = torch.zeros(3, 4, 16, dtype=b), torch.zeros(3, 2, 16, dtype=b)
    p, n = torch.zeros(3, dtype=torch.int32), torch.zeros(16)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dc.qk_norm_rotate(q, k, p, None, n, n, q, k)
    with pytest.raises(ValueError, match="queries are bfloat16"):
        dc.qk_norm_rotate(q.int(), k, p, None, n, n, q, k)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        dc.kv_append(k, k, p, p, p[None], k[None], k[None], k_norm=n)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dc.prefix_attention(q, k[None], k[None], p[None], p[:1], p[None], p, q, ws)
    with pytest.raises(dc.DCError):
        dc.linear_logprobs_workspace(3, 12, 100)
    with pytest.raises(dc.DCError):
        dc.prefix_attention_workspace(5, 2, 8, 2, 64, 100, 100)
    with pytest.raises(dc.DCError):
        dc.qk_norm_workspace(5, 2, 8, 520)
