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
# A small call's time is mostly these checks, so each reads a tensor's
# properties once, and words its refusal only when one of them is wrong.
# (get_device() is -1 for a tensor that is on no GPU.)

def _refuse_device(t, what: str, dev: int) -> None:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (got device {t.device})")
    _dc._wrong_device(what, t, dev)


def _refuse_dtype(t, what: str, dtypes) -> None:
    raise ValueError(f"{what} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")


def _vector(t, what: str, n: int, dtypes, dev: int) -> int:
    """The data pointer of a contiguous [n] tensor of one of `dtypes`."""
    if t.get_device() != dev:
        _refuse_device(t, what, dev)
    if t.dtype not in dtypes:
        _refuse_dtype(t, what, dtypes)
    if t.shape != (n,):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected ({n},)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


class _Torch:
    """What the checks use of torch, looked up once."""

    def __init__(self):
        import torch

        self.f32 = (torch.float32,)
        self.i32 = (torch.int32,)
        self.index = (torch.int64, torch.int32)
        self.i64 = torch.int64
        self.code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
        C = torch._C
        self.device = getattr(C, "_cuda_getDevice", None) or torch.cuda.current_device
        raw = getattr(C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_torch = None


def _T() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _current(t, T: _Torch) -> int:
    """The current device (-1 if `t`, the call's first tensor, is on none: the
    checks then refuse it without touching CUDA)."""
    return T.device() if t.is_cuda else -2


def _stream(stream, dev: int, T: _Torch) -> int:
    return T.stream(dev) if stream is None else _dc._stream_handle(stream)


def _matrices(ts: Sequence, what: str, rows: int, dtype, dev: int):
    """Pointers, widths and row strides of [rows, width] tensors."""
    ptrs, widths, strides = [], [], []
    for t in ts:
        shape = t.shape
        if t.get_device() != dev or t.dtype is not dtype or len(shape) != 2 or shape[0] != rows:
            r = len(ptrs)
            if t.get_device() != dev:
                _refuse_device(t, f"{what}[{r}]", dev)
            if t.dtype is not dtype:
                _refuse_dtype(t, f"{what}[{r}]", (dtype,))
            raise ValueError(f"{what}[{r}] has shape {tuple(shape)}, expected ({rows}, columns)")
        s0, s1 = t.stride()
        if s1 != 1 and shape[1] > 1:
            raise ValueError(f"{what}[{len(ptrs)}]: the vocabulary dimension must be contiguous")
        ptrs.append(t.data_ptr())
        widths.append(shape[1])
        strides.append(s0)
    return ptrs, widths, strides


def _logits(shards: Sequence, T: _Torch):
    if len(shards) == 0:
        raise ValueError("need at least one shard")
    first = shards[0]
    if first.dim() != 2:
        raise ValueError(f"shards[0] has shape {tuple(first.shape)}, expected (rows, columns)")
    dtype = first.dtype
    code = T.code.get(dtype)
    if code is None:
        raise ValueError(f"logits are bfloat16, float16 or float32 (got {dtype})")
    return first.shape[0], dtype, code, _current(first, T)


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
    T = _T()
    rows, dtype, code, dev = _logits(shards, T)
    ptrs, widths, strides = _matrices(shards, "shards", rows, dtype, dev)
    P = len(ptrs)
    top = top_lp = top_id = top64 = 0
    if top_logprobs is not None:
        top, top_lp = _alternatives(top_logprobs, "top_logprobs", rows, None, T.f32, dev)
    if top_tokens is not None:
        top, top_id = _alternatives(top_tokens, "top_tokens", rows, top if top_lp else None, T.index, dev)
        top64 = top_tokens.dtype is T.i64
    total = sum(widths)
    host = array.array("Q", ptrs + widths + strides)
    at = host.buffer_info()[0]
    f32 = T.f32
    block = _SCORE.pack(
        at, at + 8 * P, at + 16 * P, _vector(tokens, "tokens", rows, T.index, dev),
        _vector(logprobs, "logprobs", rows, f32, dev),
        0 if entropy is None else _vector(entropy, "entropy", rows, f32, dev),
        0 if lse is None else _vector(lse, "lse", rows, f32, dev), top_lp, top_id, rows,
        total if vocab is None else vocab, temperature, P, code, tokens.dtype is T.i64, top64, top, 0)
    status = _lib().dc_token_logprobs(block, _stream(stream, dev, T))
    if status:
        _dc._check(status)
    return logprobs


def _alternatives(t, what: str, rows: int, k, dtypes, dev: int):
    """k and the data pointer of a contiguous [rows, k] tensor."""
    if t.get_device() != dev:
        _refuse_device(t, what, dev)
    if t.dtype not in dtypes:
        _refuse_dtype(t, what, dtypes)
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or (k is not None and shape[1] != k) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous ({rows}, {'k' if k is None else k}) tensor (got {tuple(shape)})")
    return shape[1], t.data_ptr()


def token_logprobs_backward(shards: Sequence, tokens, lse, grad_logprobs, grads: Sequence, entropy=None,
                            grad_entropy=None, vocab: int | None = None, temperature: float = 1.0, stream=None):
    """The gradient of :func:`token_logprobs` with respect to the logits:
    ``grads[r]`` (of ``shards[r]``'s shape and type; it may be ``shards[r]``
    itself) receives that of ``sum(grad_logprobs * logprobs + grad_entropy *
    entropy)``.  ``lse`` and ``entropy`` are the forward call's outputs
    (``entropy`` only with ``grad_entropy``); the upstream gradients are
    float32 [rows], either may be None.  Padding columns receive 0.  Returns
    ``grads``."""
    T = _T()
    rows, dtype, code, dev = _logits(shards, T)
    ptrs, widths, strides = _matrices(shards, "shards", rows, dtype, dev)
    P = len(ptrs)
    if len(grads) != P:
        raise ValueError(f"need one gradient per shard (got {len(grads)} for {P})")
    gptrs, gwidths, gstrides = _matrices(grads, "grads", rows, dtype, dev)
    if gwidths != widths:
        raise ValueError("grads must have the shards' shapes")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the forward call's entropy")
    total = sum(widths)
    host = array.array("Q", ptrs + widths + strides + gptrs + gstrides)
    at = host.buffer_info()[0]
    f32 = T.f32
    block = _GRAD.pack(
        at, at + 8 * P, at + 16 * P, at + 24 * P, at + 32 * P, _vector(tokens, "tokens", rows, T.index, dev),
        _vector(lse, "lse", rows, f32, dev), 0 if entropy is None else _vector(entropy, "entropy", rows, f32, dev),
        0 if grad_logprobs is None else _vector(grad_logprobs, "grad_logprobs", rows, f32, dev),
        0 if grad_entropy is None else _vector(grad_entropy, "grad_entropy", rows, f32, dev), rows,
        total if vocab is None else vocab, temperature, P, code, tokens.dtype is T.i64, 0)
    status = _lib().dc_token_logprobs_backward(block, _stream(stream, dev, T))
    if status:
        _dc._check(status)
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

def _heads(t, what: str, shape, dtype, dev: int):
    """Pointer, token and head strides of a tensor of `shape`, (n, heads, dim);
    heads None: any number."""
    got = t.shape
    if t.get_device() != dev or t.dtype is not dtype or got != shape:
        if t.get_device() != dev:
            _refuse_device(t, what, dev)
        if t.dtype is not dtype:
            _refuse_dtype(t, what, (dtype,))
        if len(got) != 3 or got[0] != shape[0] or got[2] != shape[2] or shape[1] is not None:
            raise ValueError(f"{what} has shape {tuple(got)}, expected "
                             f"({shape[0]}, {'heads' if shape[1] is None else shape[1]}, {shape[2]})")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), s0, s1


def _cache(t, what: str, shape, dtype, dev: int):
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        if t.get_device() != dev:
            _refuse_device(t, what, dev)
        if t.dtype is not dtype:
            _refuse_dtype(t, what, (dtype,))
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    s0, s1, s2, s3 = t.stride()
    if s3 != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), s0, s1, s2


def _table(t, rows, dev: int, T: _Torch):
    """Pointer, rows, columns and row stride of a page table."""
    if t.get_device() != dev:
        _refuse_device(t, "page_table", dev)
    if t.dtype not in T.i32:
        _refuse_dtype(t, "page_table", T.i32)
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows):
        raise ValueError(f"page_table has shape {tuple(shape)}, expected ({'sequences' if rows is None else rows}, pages)")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError("page_table: rows must be contiguous")
    return t.data_ptr(), shape[0], shape[1], s0


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
    T = _T()
    dtype = k.dtype
    code = T.code.get(dtype)
    if code is None:
        raise ValueError(f"keys are bfloat16, float16 or float32 (got {dtype})")
    dev = _current(k, T)
    shape = k.shape
    if len(shape) != 3:
        raise ValueError(f"k has shape {tuple(shape)}, expected (tokens, heads, dim)")
    n, hk, d = shape
    kp, k0, k1 = _heads(k, "k", shape, dtype, dev)
    vp, v0, v1 = _heads(v, "v", shape, dtype, dev)
    hq = qp = q0 = q1 = op = o0 = o1 = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        qp, q0, q1 = _heads(q, "q", (n, None, d), dtype, dev)
        hq = q.shape[1]
        op, o0, o1 = _heads(q_out, "q_out", (n, hq, d), dtype, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rot = cos_rows = cs = 0
    if cos_sin is not None:
        if cos_sin.get_device() != dev:
            _refuse_device(cos_sin, "cos_sin", dev)
        if cos_sin.dtype not in T.f32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError(f"cos_sin must be a contiguous float32 (positions, rotary_dim) tensor "
                             f"(got {cos_sin.dtype} {tuple(cos_sin.shape)})")
        cos_rows, rot = cos_sin.shape
        cs = cos_sin.data_ptr()
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != hk or shape[3] != d:
        raise ValueError(f"k_cache has shape {tuple(shape)}, expected (pages, page size, {hk}, {d})")
    table, table_rows, table_width, table_stride = _table(page_table, None, dev, T)
    block = _APPEND.pack(
        qp, kp, vp, op, _vector(positions, "positions", n, T.i32, dev), _vector(seqs, "seqs", n, T.i32, dev), table, cs,
        *_cache(k_cache, "k_cache", shape, dtype, dev), *_cache(v_cache, "v_cache", shape, dtype, dev), q0, q1, k0, k1,
        v0, v1, o0, o1, n, table_rows, table_width, table_stride, cos_rows, shape[0], shape[1], hq, hk, d, rot,
        1 if interleaved else 0, code, 0)
    status = _lib().dc_kv_append(block, _stream(stream, dev, T))
    if status:
        _dc._check(status)
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
    T = _T()
    dtype = q.dtype
    code = T.code.get(dtype)
    if code is None or code == 2:
        raise ValueError(f"queries are bfloat16 or float16 (got {dtype})")
    dev = _current(q, T)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q has shape {tuple(shape)}, expected (sequences, heads, dim)")
    n, hq, d = shape
    qp, q0, q1 = _heads(q, "q", shape, dtype, dev)
    op, o0, o1 = _heads(out, "out", shape, dtype, dev)
    cache = k_cache.shape
    if len(cache) != 4 or cache[3] != d:
        raise ValueError(f"k_cache has shape {tuple(cache)}, expected (pages, page size, heads, {d})")
    table, _, table_width, table_stride = _table(page_table, n, dev, T)
    lse_ptr = 0
    if lse is not None:
        if lse.get_device() != dev:
            _refuse_device(lse, "lse", dev)
        if lse.dtype not in T.f32 or lse.shape != (n, hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 ({n}, {hq}) tensor (got {lse.dtype} {tuple(lse.shape)})")
        lse_ptr = lse.data_ptr()
    if workspace.get_device() != dev:
        _refuse_device(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    block = _ATTEND.pack(
        qp, op, lse_ptr, table, _vector(lengths, "lengths", n, T.i32, dev), workspace.data_ptr(), workspace.nbytes,
        *_cache(k_cache, "k_cache", cache, dtype, dev), *_cache(v_cache, "v_cache", cache, dtype, dev), q0, q1, o0, o1,
        n, table_width, table_stride, cache[0], cache[1], hq, cache[2], d, window, code,
        d ** -0.5 if scale is None else scale, 0)
    status = _lib().dc_paged_attention(block, _stream(stream, dev, T))
    if status:
        _dc._check(status)
    return out
