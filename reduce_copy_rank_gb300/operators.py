"""Operators of language models beside the collectives: log probabilities over
vocabulary shards and their gradient, the paged key-value cache and the
attention of single new tokens over it.

A thin binding like the rest of the package: tensors become pointers, sizes
and strides in the argument blocks of ``include/dc.h``, and the work runs in
the library's CUDA kernels, one launch a call.  A row's or a sequence's
result depends on nothing else in the call: the same bits in a batch of one
and of a thousand, and, for the log probabilities, under every sharding.
"""
from __future__ import annotations

import array
import ctypes
import math
import struct
from typing import Sequence

import reduce_copy_rank_gb300 as _dc

MAX_TOP = 32
MAX_VOCAB = 1 << 22
ATTENTION_DIMS = (64, 96, 128, 192, 256)


class _Block:
    """The layout of an argument block of include/dc.h."""

    def __init__(self, layout: str, names: str):
        self.pack = struct.Struct("@" + layout).pack
        self.names = names.split()

    def of(self, fields: dict) -> bytes:
        unknown = set(fields) - set(self.names)
        if unknown:
            raise TypeError(f"unknown argument(s): {sorted(unknown)}")
        return self.pack(*(fields.get(n, 0) for n in self.names))


_SCORE = _Block("9Q2qd6i", "shards widths row_strides tokens logprobs entropy lse top_logprobs top_tokens "
                           "rows vocab temperature ranks dtype tokens_64 top_tokens_64 top reserved")
_GRAD = _Block("10Q2qd4i", "shards widths row_strides grads grad_row_strides tokens lse entropy grad_logprobs "
                           "grad_entropy rows vocab temperature ranks dtype tokens_64 reserved")
_CACHES = "k_cache k_page_stride k_slot_stride k_cache_head_stride v_cache v_page_stride v_slot_stride " \
          "v_cache_head_stride "
_APPEND = _Block("24Q6q8i", "q k v q_out positions seqs page_table cos_sin " + _CACHES +
                 "q_token_stride q_head_stride k_token_stride k_head_stride v_token_stride v_head_stride "
                 "q_out_token_stride q_out_head_stride tokens table_rows table_width table_stride cos_sin_rows "
                 "num_pages page_size q_heads kv_heads dim rotary_dim interleaved dtype reserved")
_ATTEND = _Block("19Q4q6ifi", "q out lse page_table lengths workspace workspace_bytes " + _CACHES +
                 "q_seq_stride q_head_stride out_seq_stride out_head_stride seqs table_width table_stride num_pages "
                 "page_size q_heads kv_heads dim window dtype scale reserved")

_bound = None


def _lib():
    """The library with these functions' signatures set."""
    global _bound
    if _bound is None:
        L = _dc.lib()
        for f in ("dc_token_logprobs", "dc_token_logprobs_backward", "dc_kv_append", "dc_paged_attention"):
            getattr(L, f).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            getattr(L, f).restype = ctypes.c_int
        L.dc_attention_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_int64]
        L.dc_attention_workspace_bytes.restype = ctypes.c_size_t
        _bound = L
    return _bound


# ------------------------------------------------------------ raw (C ABI) ---
# The argument blocks of include/dc.h by field name (fields left out are 0;
# the caches' strides are k_page_stride, k_slot_stride, k_cache_head_stride and
# the same for v).  Pointers are ints; host arrays (shards, widths, strides)
# are passed as sequences.  They return the status instead of raising.

def _with_arrays(block: _Block, fields: dict, keep: list) -> bytes:
    f = dict(fields)
    for name in ("shards", "widths", "row_strides", "grads", "grad_row_strides"):
        if name in f and not isinstance(f[name], int):
            keep.append(array.array("Q", f[name]))
            f[name] = keep[-1].buffer_info()[0]
    return block.of(f)


def dc_token_logprobs(stream: int = 0, **fields) -> int:
    keep = []
    return _lib().dc_token_logprobs(_with_arrays(_SCORE, fields, keep), stream)


def dc_token_logprobs_backward(stream: int = 0, **fields) -> int:
    keep = []
    return _lib().dc_token_logprobs_backward(_with_arrays(_GRAD, fields, keep), stream)


def dc_kv_append(stream: int = 0, **fields) -> int:
    return _lib().dc_kv_append(_APPEND.of(fields), stream)


def dc_paged_attention(stream: int = 0, **fields) -> int:
    return _lib().dc_paged_attention(_ATTEND.of(fields), stream)


def dc_attention_workspace_bytes(seqs: int, q_heads: int, kv_heads: int, dim: int, max_tokens: int) -> int:
    return int(_lib().dc_attention_workspace_bytes(seqs, q_heads, kv_heads, dim, max_tokens))


# ------------------------------------------------------------ tensor checks ---

def _on_device(t, what: str, dev: int) -> None:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (got device {t.device})")
    if t.get_device() != dev:
        _dc._wrong_device(what, t, dev)


def _vector(t, what: str, n: int, dtypes, dev: int) -> int:
    """The data pointer of a contiguous [n] tensor of one of `dtypes`."""
    if not t.is_cuda or t.get_device() != dev:
        _on_device(t, what, dev)
    if t.dtype not in dtypes:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected ({n},)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


_types = None


def _T():
    """torch's element types that the operators take."""
    global _types
    if _types is None:
        import torch

        class _types:  # noqa: N801
            f32 = (torch.float32,)
            i32 = (torch.int32,)
            index = (torch.int64, torch.int32)
            i64 = torch.int64
            code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    return _types


def _matrices(ts: Sequence, what: str, rows: int, dtype, dev: int):
    """Pointers, widths and row strides of [rows, width] tensors."""
    ptrs, widths, strides = [], [], []
    for r, t in enumerate(ts):
        if not t.is_cuda or t.get_device() != dev:
            _on_device(t, f"{what}[{r}]", dev)
        if t.dtype is not dtype:
            raise ValueError(f"{what}[{r}] has dtype {t.dtype}, expected {dtype}")
        shape = t.shape
        if len(shape) != 2 or shape[0] != rows:
            raise ValueError(f"{what}[{r}] has shape {tuple(shape)}, expected ({rows}, columns)")
        s0, s1 = t.stride()
        if s1 != 1 and shape[1] > 1:
            raise ValueError(f"{what}[{r}]: the vocabulary dimension must be contiguous")
        ptrs.append(t.data_ptr())
        widths.append(shape[1])
        strides.append(s0)
    return array.array("Q", ptrs), array.array("Q", widths), array.array("Q", strides)


def _logits(shards: Sequence):
    if len(shards) == 0:
        raise ValueError("need at least one shard")
    first = shards[0]
    if first.dim() != 2:
        raise ValueError(f"shards[0] has shape {tuple(first.shape)}, expected (rows, columns)")
    code = _T().code.get(first.dtype)
    if code is None:
        raise ValueError(f"logits are bfloat16, float16 or float32 (got {first.dtype})")
    dev = _dc._cur_dev() if first.is_cuda else -1
    return first.shape[0], code, dev


# ------------------------------------------------------- log probabilities ---

def token_logprobs(shards: Sequence, tokens, logprobs, entropy=None, lse=None, top_logprobs=None, top_tokens=None,
                   vocab: int | None = None, temperature: float = 1.0, stream=None):
    """Log probabilities of given tokens under logits held as P vocabulary
    shards (``shards[r]``: [rows, columns of rank r], bfloat16, float16 or
    float32; any row stride), without gathering them.

    ``logprobs[i]`` (float32) receives the log probability of ``tokens[i]``
    (int32 or int64) under ``softmax(logits[i] / temperature)`` over the first
    ``vocab`` columns (default: all; later ones are padding).  Optional
    outputs: ``entropy`` and ``lse`` (the log of the normaliser), float32
    [rows]; ``top_logprobs`` (float32) and ``top_tokens`` (int32 or int64),
    [rows, k] with k <= 32: the k largest logits, ties to the lowest index.

    A negative token is not scored (its entry is 0), a token past the
    vocabulary gives NaN.  Logits of -inf have probability 0; a row of
    nothing else gives -inf.  Bits depend on the row alone: not on the other
    rows, the number of shards or where they are cut.  Returns ``logprobs``."""
    rows, code, dev = _logits(shards)
    ptrs, widths, strides = _matrices(shards, "shards", rows, shards[0].dtype, dev)
    T = _T()
    top = 0
    top_lp = top_id = top64 = 0
    for name, t, types in (("top_logprobs", top_logprobs, T.f32), ("top_tokens", top_tokens, T.index)):
        if t is None:
            continue
        _on_device(t, name, dev)
        if t.dtype not in types:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in types)}")
        if t.dim() != 2 or t.shape[0] != rows or (top and t.shape[1] != top) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous ({rows}, {top or 'k'}) tensor (got {tuple(t.shape)})")
        top = t.shape[1]
        if name == "top_tokens":
            top_id, top64 = t.data_ptr(), int(t.dtype is T.i64)
        else:
            top_lp = t.data_ptr()
    block = _SCORE.pack(
        ptrs.buffer_info()[0], widths.buffer_info()[0], strides.buffer_info()[0],
        _vector(tokens, "tokens", rows, T.index, dev), _vector(logprobs, "logprobs", rows, T.f32, dev),
        0 if entropy is None else _vector(entropy, "entropy", rows, T.f32, dev),
        0 if lse is None else _vector(lse, "lse", rows, T.f32, dev), top_lp, top_id, rows,
        sum(widths) if vocab is None else vocab, temperature, len(ptrs), code, int(tokens.dtype is T.i64), top64, top, 0)
    _dc._check(_lib().dc_token_logprobs(block, _dc._stream_handle(stream)))
    return logprobs


def token_logprobs_backward(shards: Sequence, tokens, lse, grad_logprobs, grads: Sequence, entropy=None,
                            grad_entropy=None, vocab: int | None = None, temperature: float = 1.0, stream=None):
    """The gradient of :func:`token_logprobs` with respect to the logits:
    ``grads[r]`` (of ``shards[r]``'s shape and type; it may be ``shards[r]``
    itself) receives that of ``sum(grad_logprobs * logprobs + grad_entropy *
    entropy)``.  ``lse`` and ``entropy`` are the forward call's outputs
    (``entropy`` only with ``grad_entropy``); the upstream gradients are
    float32 [rows], either may be None.  Padding columns receive 0.  Returns
    ``grads``."""
    rows, code, dev = _logits(shards)
    dtype = shards[0].dtype
    ptrs, widths, strides = _matrices(shards, "shards", rows, dtype, dev)
    if len(grads) != len(shards):
        raise ValueError(f"need one gradient per shard (got {len(grads)} for {len(shards)})")
    gptrs, gwidths, gstrides = _matrices(grads, "grads", rows, dtype, dev)
    if gwidths != widths:
        raise ValueError("grads must have the shards' shapes")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the forward call's entropy")
    T = _T()
    block = _GRAD.pack(
        ptrs.buffer_info()[0], widths.buffer_info()[0], strides.buffer_info()[0], gptrs.buffer_info()[0],
        gstrides.buffer_info()[0], _vector(tokens, "tokens", rows, T.index, dev), _vector(lse, "lse", rows, T.f32, dev),
        0 if entropy is None else _vector(entropy, "entropy", rows, T.f32, dev),
        0 if grad_logprobs is None else _vector(grad_logprobs, "grad_logprobs", rows, T.f32, dev),
        0 if grad_entropy is None else _vector(grad_entropy, "grad_entropy", rows, T.f32, dev), rows,
        sum(widths) if vocab is None else vocab, temperature, len(ptrs), code, int(tokens.dtype is T.i64), 0)
    _dc._check(_lib().dc_token_logprobs_backward(block, _dc._stream_handle(stream)))
    return grads


_function = None


def logprobs_and_entropy(shards: Sequence, tokens, vocab: int | None = None, temperature: float = 1.0):
    """``(logprobs, entropy)`` of :func:`token_logprobs` as new tensors that
    autograd differentiates with respect to every shard (through
    :func:`token_logprobs_backward`)."""
    global _function
    import torch

    if _function is None:
        class TokenLogprobs(torch.autograd.Function):
            @staticmethod
            def forward(ctx, tokens, vocab, temperature, *shards):
                rows = shards[0].shape[0]
                logprobs, entropy, lse = (torch.empty(rows, dtype=torch.float32, device=shards[0].device)
                                          for _ in range(3))
                token_logprobs(shards, tokens, logprobs, entropy=entropy, lse=lse, vocab=vocab, temperature=temperature)
                ctx.save_for_backward(tokens, lse, entropy, *shards)
                ctx.vocab, ctx.temperature = vocab, temperature
                return logprobs, entropy

            @staticmethod
            def backward(ctx, g, h):
                tokens, lse, entropy, *shards = ctx.saved_tensors
                grads = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in shards]
                # upstream gradients may be broadcast (a sum's is one number for all rows)
                g, h = (None if u is None else u.to(torch.float32).contiguous() for u in (g, h))
                token_logprobs_backward(shards, tokens, lse, g, grads, entropy=entropy, grad_entropy=h,
                                        vocab=ctx.vocab, temperature=ctx.temperature)
                return (None, None, None, *grads)

        _function = TokenLogprobs
    return _function.apply(tokens, vocab, temperature, *shards)


# ------------------------------------------------------------ paged cache ---

def _heads(t, what: str, n: int, dtype, dev: int):
    """Pointer, token and head strides of a [n, heads, dim] tensor."""
    if not t.is_cuda or t.get_device() != dev:
        _on_device(t, what, dev)
    if t.dtype is not dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != n:
        raise ValueError(f"{what} has shape {tuple(shape)}, expected ({n}, heads, dim)")
    st = t.stride()
    if st[2] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), st[0], st[1]


def _cache(t, what: str, shape, dtype, dev: int):
    if not t.is_cuda or t.get_device() != dev:
        _on_device(t, what, dev)
    if t.dtype is not dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected "
                         f"{'(pages, page size, heads, dim)' if shape is None else tuple(shape)}")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), st[0], st[1], st[2]


def _table(t, rows, dev: int):
    if not t.is_cuda or t.get_device() != dev:
        _on_device(t, "page_table", dev)
    if t.dtype not in _T().i32:
        raise ValueError(f"page_table has dtype {t.dtype}, expected torch.int32")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"page_table has shape {tuple(t.shape)}, expected ({'sequences' if rows is None else rows}, pages)")
    st = t.stride()
    if st[1] != 1 and t.shape[1] > 1:
        raise ValueError("page_table: rows must be contiguous")
    return t.data_ptr(), st[0]


def kv_append(k, v, positions, seqs, page_table, k_cache, v_cache, q=None, q_out=None, cos_sin=None,
              interleaved: bool = False, stream=None):
    """Puts the keys and values of new tokens ([tokens, kv_heads, dim]) into a
    paged cache ([pages, page_size, kv_heads, dim] tensors, or views of that
    shape with any strides), rotating the keys, and the queries ``q`` into
    ``q_out`` ([tokens, q_heads, dim]; ``q_out`` may be ``q``), to their
    positions.  Token i of sequence ``seqs[i]`` at ``positions[i]`` (int32)
    goes to slot ``positions[i] % page_size`` of page ``page_table[seqs[i],
    positions[i] // page_size]`` (int32).

    ``cos_sin`` (float32 [positions, rotary_dim]): the cosines of a position's
    rotary_dim/2 angles, then their sines; None: no rotation.  Pair j is
    elements j and j + rotary_dim/2, or 2j and 2j + 1 if ``interleaved``;
    elements past rotary_dim stay.

    A negative position is padding and writes nothing.  A token whose
    sequence, position or page does not exist writes no cache; its queries
    become NaN.  Returns ``q_out``."""
    dtype = k.dtype
    code = _T().code.get(dtype)
    if code is None:
        raise ValueError(f"keys are bfloat16, float16 or float32 (got {dtype})")
    dev = _dc._cur_dev() if k.is_cuda else -1
    if k.dim() != 3:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected (tokens, heads, dim)")
    n, hk, d = k.shape
    kp = _heads(k, "k", n, dtype, dev)
    vp = _heads(v, "v", n, dtype, dev)
    if v.shape != k.shape:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {tuple(k.shape)}")
    hq, qp, op = 0, (0, 0, 0), (0, 0, 0)
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        qp, op = _heads(q, "q", n, dtype, dev), _heads(q_out, "q_out", n, dtype, dev)
        hq = q.shape[1]
        if q.shape[2] != d or q_out.shape != q.shape:
            raise ValueError(f"q and q_out have shapes {tuple(q.shape)} and {tuple(q_out.shape)}, expected ({n}, heads, {d})")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rot, cos_rows, cs = 0, 0, 0
    if cos_sin is not None:
        _on_device(cos_sin, "cos_sin", dev)
        if cos_sin.dtype not in _T().f32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError(f"cos_sin must be a contiguous float32 (positions, rotary_dim) tensor "
                             f"(got {cos_sin.dtype} {tuple(cos_sin.shape)})")
        cos_rows, rot = cos_sin.shape
        cs = cos_sin.data_ptr()
    kc = _cache(k_cache, "k_cache", None, dtype, dev)
    shape = k_cache.shape
    if shape[2] != hk or shape[3] != d:
        raise ValueError(f"k_cache has shape {tuple(shape)}, expected (pages, page size, {hk}, {d})")
    vc = _cache(v_cache, "v_cache", shape, dtype, dev)
    T = _T()
    table, table_stride = _table(page_table, None, dev)
    block = _APPEND.pack(
        qp[0], kp[0], vp[0], op[0], _vector(positions, "positions", n, T.i32, dev), _vector(seqs, "seqs", n, T.i32, dev),
        table, cs, *kc, *vc, qp[1], qp[2], kp[1], kp[2], vp[1], vp[2], op[1], op[2], n, page_table.shape[0],
        page_table.shape[1], table_stride, cos_rows, shape[0], shape[1], hq, hk, d, rot, int(interleaved), code, 0)
    _dc._check(_lib().dc_kv_append(block, _dc._stream_handle(stream)))
    return q_out


def attention_workspace(seqs: int, q_heads: int, kv_heads: int, dim: int, max_tokens: int, device=None):
    """A zeroed workspace tensor for :func:`paged_attention` with up to
    ``seqs`` sequences and page tables of up to ``max_tokens`` tokens a row
    (allocated by torch; the library itself allocates nothing).  Keep it: a
    call leaves it ready for the next.  One workspace per stream."""
    import torch

    n = dc_attention_workspace_bytes(seqs, q_heads, kv_heads, dim, max_tokens)
    if n == 0:
        raise _dc.DCError(1, _dc.last_error() or "no such attention")
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def paged_attention(q, k_cache, v_cache, page_table, lengths, out, workspace, scale: float | None = None,
                    window: int = 0, lse=None, stream=None):
    """Attention of one new token per sequence over a paged cache.

    ``q``, ``out``: [sequences, q_heads, dim] (bfloat16 or float16; dim 64,
    96, 128, 192 or 256); caches as in :func:`kv_append`, q_heads a multiple
    of kv_heads; ``page_table`` int32 [sequences, pages], ``lengths`` int32
    [sequences]: sequence b attends to its first ``lengths[b]`` tokens, or to
    the last ``window`` of them.  ``scale``: default ``dim ** -0.5``.  ``lse``
    (float32 [sequences, q_heads]) receives the log of the normaliser, with
    which results over parts of a context can be joined.

    A length of 0 gives zeros (lse -inf).  A page number outside the cache, or
    a length past the table, gives NaN.  ``workspace``: see
    :func:`attention_workspace`.  Returns ``out``."""
    dtype = q.dtype
    code = _T().code.get(dtype)
    if code is None or code == 2:
        raise ValueError(f"queries are bfloat16 or float16 (got {dtype})")
    dev = _dc._cur_dev() if q.is_cuda else -1
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected (sequences, heads, dim)")
    n, hq, d = q.shape
    qp = _heads(q, "q", n, dtype, dev)
    op = _heads(out, "out", n, dtype, dev)
    if out.shape != q.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
    kc = _cache(k_cache, "k_cache", None, dtype, dev)
    shape = k_cache.shape
    if shape[3] != d:
        raise ValueError(f"k_cache has shape {tuple(shape)}, expected (pages, page size, heads, {d})")
    vc = _cache(v_cache, "v_cache", shape, dtype, dev)
    T = _T()
    table, table_stride = _table(page_table, n, dev)
    lse_ptr = 0
    if lse is not None:
        _on_device(lse, "lse", dev)
        if lse.dtype not in T.f32 or lse.shape != q.shape[:2] or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 ({n}, {hq}) tensor (got {lse.dtype} {tuple(lse.shape)})")
        lse_ptr = lse.data_ptr()
    if not workspace.is_cuda or workspace.get_device() != dev or not workspace.is_contiguous():
        _on_device(workspace, "workspace", dev)
        raise ValueError("workspace must be contiguous")
    block = _ATTEND.pack(
        qp[0], op[0], lse_ptr, table, _vector(lengths, "lengths", n, T.i32, dev), workspace.data_ptr(), workspace.nbytes,
        *kc, *vc, qp[1], qp[2], op[1], op[2], n, page_table.shape[1], table_stride, shape[0], shape[1], hq, shape[2], d,
        window, code, 1.0 / math.sqrt(d) if scale is None else scale, 0)
    _dc._check(_lib().dc_paged_attention(block, _dc._stream_handle(stream)))
    return out
