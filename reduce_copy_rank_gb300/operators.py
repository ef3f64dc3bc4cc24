"""Operators of language models beside the collectives: log probabilities over
vocabulary shards and their gradient, the paged key-value cache and the
attention of single new tokens over it.

A thin binding like the rest of the package: tensors become pointers, sizes
and strides in the argument blocks of ``include/dc.h`` (read by the extension
module ``_binding``, whose checks raise ``ValueError``), and the work runs in
the library's CUDA kernels, one launch a call.  A row's or a sequence's
result depends on nothing else in the call: the same bits in a batch of one
and of a thousand, and, for the log probabilities, under every sharding.
What a call has written counts as changed in place: where autograd had kept
those numbers for a gradient, that gradient raises.
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


# ------------------------------------------------------------ tensor API ---

_module = None


def _binding():
    """The extension module that reads the tensors, bound to the library."""
    global _module
    if _module is None:
        L = _lib()
        import torch  # noqa: F401  (its libraries first)

        try:
            from . import _binding as module
        except ImportError as e:
            raise _dc.LibraryMissing(f"the extension module _binding cannot be loaded ({e}): build it with `python -m "
                                     "reduce_copy_rank_gb300._build` or __graft_entry__.build()") from e
        module.bind(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "dc_token_logprobs", "dc_token_logprobs_backward", "dc_kv_append", "dc_paged_attention")))
        _module = module
    return _module


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
    status = (_module or _binding()).token_logprobs(shards, tokens, logprobs, entropy, lse, top_logprobs, top_tokens, vocab,
                                                    temperature, stream)
    if status:
        _dc._check(status)
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
    status = (_module or _binding()).token_logprobs_backward(shards, tokens, lse, grad_logprobs, grads, entropy,
                                                             grad_entropy, vocab, temperature, stream)
    if status:
        _dc._check(status)
    return grads


_function = None


def logprobs_and_entropy(shards: Sequence, tokens, vocab: int | None = None, temperature: float = 1.0):
    """``(logprobs, entropy)`` of :func:`token_logprobs` as new tensors that
    autograd differentiates with respect to every shard (through
    :func:`token_logprobs_backward`, which computes every shard's gradient,
    wanted or not), once: a second derivative raises."""
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
                ctx.set_materialize_grads(False)  # an output that is not used has no upstream gradient to read
                ctx.save_for_backward(tokens, lse, entropy, *shards)
                ctx.vocab, ctx.temperature = vocab, temperature
                return logprobs, entropy

            @staticmethod
            def backward(ctx, g, h):
                tokens, lse, entropy, *shards = ctx.saved_tensors
                if g is None and h is None:
                    return (None,) * (3 + len(shards))
                grads = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in shards]
                # upstream gradients may be broadcast (a sum's is one number for all rows)
                g, h = (None if u is None else u.to(torch.float32).contiguous() for u in (g, h))
                token_logprobs_backward(shards, tokens, lse, g, grads, entropy=entropy, grad_entropy=h,
                                        vocab=ctx.vocab, temperature=ctx.temperature)
                if torch.is_grad_enabled():  # create_graph: the gradients leave a kernel, no graph holds them
                    grads = FirstDerivative.apply(len(grads), *grads, *shards, *(u for u in (g, h) if u is not None))
                return (None, None, None, *grads)

        class FirstDerivative(torch.autograd.Function):
            """The gradients, with the tensors that they depend on: their own derivative is refused."""

            @staticmethod
            def forward(ctx, count, *tensors):
                return tuple(t.detach() for t in tensors[:count])

            @staticmethod
            def backward(ctx, *_):
                raise RuntimeError("logprobs_and_entropy has no second derivative: its gradients cannot be differentiated")

        _function = TokenLogprobs
    return _function.apply(tokens, vocab, temperature, *shards)


# ------------------------------------------------------------ paged cache ---

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
    status = (_module or _binding()).kv_append(k, v, positions, seqs, page_table, k_cache, v_cache, q, q_out, cos_sin,
                                               interleaved, stream)
    if status:
        _dc._check(status)
    return q_out


def attention_workspace(seqs: int, q_heads: int, kv_heads: int, dim: int, max_tokens: int, device=None):
    """A zeroed workspace tensor for :func:`paged_attention` with up to
    ``seqs`` sequences and page tables of up to ``max_tokens`` tokens a row
    (allocated by torch; the library itself allocates nothing).  Keep it: a
    call leaves it, and any part of it that starts where it does, ready for
    the next.  One workspace per stream."""
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
    status = (_module or _binding()).paged_attention(q, k_cache, v_cache, page_table, lengths, out, workspace, scale, window,
                                                     lse, stream)
    if status:
        _dc._check(status)
    return out
